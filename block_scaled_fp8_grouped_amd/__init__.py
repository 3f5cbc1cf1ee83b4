"""Block-scaled FP8 grouped quantize / wgrad / fprop for MoE expert layers on MI355X (gfx950).

Thin ctypes binding of ``libbsfp8.so``.  It only marshals arguments: tensor data pointers,
sizes and torch's current HIP stream go to the C ABI declared in ``include/bsfp8.h``; every
step of the computation runs in the library's kernels.  PyTorch supplies device memory and the
stream.  If the library has not been built, importing works but every call raises.

Functions keep the C names without the ``bsfp8_`` prefix:
  grouped_quantize, grouped_gemm_wgrad, grouped_gemm_fprop, the size queries, strerror; and the steps around them:
  grouped_gemm_swiglu, residual_norm, adamw_step, route_topk, dispatch_plan, dispatch, dispatch_quantize, combine,
  grouped_act_checkpoint and their gradients.
``alloc_quantized`` and ``alloc_*`` helpers size output tensors with the library's own size
queries.
"""
import ctypes
import importlib
import os
import warnings

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libbsfp8.so")

RECIPE_MX = 1  # BSFP8_RECIPE_MX_1X32_E8M0
RECIPE_PC = 2  # BSFP8_RECIPE_PER_CHANNEL_128_F32
RECIPE_MX4 = 3  # BSFP8_RECIPE_MXFP4_1X32_E8M0
GEMM_FP8_MFMA = 0x100  # BSFP8_GEMM_FP8_MFMA: OR into RECIPE_MX for the GEMMs on the scaled fp8 MFMA
ROWWISE = 1
COLWISE = 2
ACT_SRELU = 1  # BSFP8_ACT_SRELU: y = p * max(h, 0)^2
ACT_SRELU_GRAD = 2  # BSFP8_ACT_SRELU_GRAD: g = dy * p * 2 max(h, 0)
ACT_SWIGLU = 3  # BSFP8_ACT_SWIGLU: y = p * silu(a) * b, h = (a | b)
ACT_SWIGLU_GRAD = 4  # BSFP8_ACT_SWIGLU_GRAD: (da | db) of the scaled SwiGLU
OUT_F32 = 0
OUT_BF16 = 1
STATUS_NEGATIVE_SPLIT = 1
STATUS_EXCEEDS_CAPACITY = 2
MAX_GROUPS = 1024
F32 = 0  # BSFP8_F32
BF16 = 1  # BSFP8_BF16
GATE_NONE = 0
GATE_CHANNEL = 1  # gate[cols]
GATE_TOKEN = 2  # gate[rows]
STATE_F32 = 0
STATE_8BIT = 1
ROUTE_SOFTMAX = 1  # BSFP8_ROUTE_SOFTMAX: scores of softmax(logits)
ROUTE_SIGMOID = 2  # BSFP8_ROUTE_SIGMOID: scores of sigmoid(logits)
MAX_TOP_K = 32

_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_vp = ctypes.c_void_p
_sz = ctypes.c_size_t

_lib = None


class BSFP8Error(RuntimeError):
    pass


def lib():
    """The loaded libbsfp8.so; raises when it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise BSFP8Error(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                             "(or python -m block_scaled_fp8_grouped_amd._build)")
        L = ctypes.CDLL(LIB_PATH)
        L.bsfp8_colwise_rows_bound.restype = _i64
        L.bsfp8_colwise_rows_bound.argtypes = [_i64, _i32]
        L.bsfp8_colwise_data_bytes.restype = _sz
        L.bsfp8_colwise_data_bytes.argtypes = [_i64, _i64, _i32, ctypes.c_int]
        L.bsfp8_colwise_scale_bytes.restype = _sz
        L.bsfp8_colwise_scale_bytes.argtypes = [_i64, _i64, _i32, ctypes.c_int]
        L.bsfp8_rowwise_data_bytes.restype = _sz
        L.bsfp8_rowwise_data_bytes.argtypes = [_i64, _i64, ctypes.c_int]
        L.bsfp8_rowwise_scale_bytes.restype = _sz
        L.bsfp8_rowwise_scale_bytes.argtypes = [_i64, _i64]
        L.bsfp8_grouped_quantize.restype = ctypes.c_int
        L.bsfp8_grouped_quantize.argtypes = [_vp, _i64, _i64, _vp, _i32, ctypes.c_int, ctypes.c_int,
                                             ctypes.c_float, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
        L.bsfp8_grouped_act_quantize.restype = ctypes.c_int
        L.bsfp8_grouped_act_quantize.argtypes = [ctypes.c_int, _vp, _vp, _vp, _i64, _i64, _vp, _i32, ctypes.c_int,
                                                 ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp]
        L.bsfp8_grouped_gemm_wgrad.restype = ctypes.c_int
        L.bsfp8_grouped_gemm_wgrad.argtypes = [_vp, _vp, _i64, _vp, _vp, _i64, _vp, _i32, _i64, ctypes.c_int,
                                               _vp, ctypes.c_int, _vp, _vp]
        L.bsfp8_grouped_gemm_fprop.restype = ctypes.c_int
        L.bsfp8_grouped_gemm_fprop.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _i32, ctypes.c_int, _vp,
                                               ctypes.c_int, _vp, _vp]
        L.bsfp8_grouped_gemm_dgrad.restype = ctypes.c_int
        L.bsfp8_grouped_gemm_dgrad.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _i32, ctypes.c_int, _vp,
                                               ctypes.c_int, _vp, _vp]
        L.bsfp8_grouped_gemm_swiglu.restype = ctypes.c_int
        L.bsfp8_grouped_gemm_swiglu.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _i32, ctypes.c_int, _vp,
                                                _vp, ctypes.c_int, ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp]
        L.bsfp8_grouped_gemm_swiglu_grad_workspace_bytes.restype = _sz
        L.bsfp8_grouped_gemm_swiglu_grad_workspace_bytes.argtypes = [_i64, _i64, _i32]
        L.bsfp8_grouped_gemm_swiglu_grad.restype = ctypes.c_int
        L.bsfp8_grouped_gemm_swiglu_grad.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _vp, _i32,
                                                     ctypes.c_int, _vp, ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp,
                                                     _vp, _vp]
        _f, _d = ctypes.c_float, ctypes.c_double
        L.bsfp8_residual_norm.restype = ctypes.c_int
        L.bsfp8_residual_norm.argtypes = [_i64, _i64, _vp, ctypes.c_int, _vp, _vp, _vp, _vp, ctypes.c_int, _f, _f, _f,
                                          _f, _vp, _vp, _vp, _vp, _vp]
        L.bsfp8_residual_norm_grad_workspace_bytes.restype = _sz
        L.bsfp8_residual_norm_grad_workspace_bytes.argtypes = [_i64, _i64]
        L.bsfp8_residual_norm_grad.restype = ctypes.c_int
        L.bsfp8_residual_norm_grad.argtypes = [_i64, _i64, ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                               ctypes.c_int, _f, _f, _f, _vp, _vp, _vp, _vp, _vp, ctypes.c_int, _vp,
                                               _vp]
        L.bsfp8_adamw_plan_bytes.restype = _sz
        L.bsfp8_adamw_plan_bytes.argtypes = [_vp, _i32, ctypes.POINTER(_i64)]
        L.bsfp8_adamw_plan.restype = ctypes.c_int
        L.bsfp8_adamw_plan.argtypes = [_vp, _i32, ctypes.c_int, ctypes.c_int, ctypes.c_int, _vp, _sz]
        L.bsfp8_adamw_step.restype = ctypes.c_int
        L.bsfp8_adamw_step.argtypes = [_vp, _i32, _i64, ctypes.c_int, ctypes.c_int, ctypes.c_int, _d, _d, _d, _d, _d,
                                       _i64, _vp, _vp, _vp, _vp, _vp]
        L.bsfp8_adamw_step_stochastic.restype = ctypes.c_int
        L.bsfp8_adamw_step_stochastic.argtypes = L.bsfp8_adamw_step.argtypes[:-1] + [ctypes.c_uint64, _vp]
        L.bsfp8_route_topk_workspace_bytes.restype = _sz
        L.bsfp8_route_topk_workspace_bytes.argtypes = [_i64, _i32]
        L.bsfp8_route_topk.restype = ctypes.c_int
        L.bsfp8_route_topk.argtypes = [_vp, ctypes.c_int, _i64, _i32, _i32, ctypes.c_int, _vp, ctypes.c_int, _f, _vp, _vp,
                                       _vp, _vp, _vp]
        L.bsfp8_route_topk_grad.restype = ctypes.c_int
        L.bsfp8_route_topk_grad.argtypes = [_vp, _vp, ctypes.c_int, _vp, _i64, _i32, _i32, ctypes.c_int, ctypes.c_int, _f,
                                            _vp, _vp, _vp]
        L.bsfp8_dispatch_plan_workspace_bytes.restype = _sz
        L.bsfp8_dispatch_plan_workspace_bytes.argtypes = [_i64, _i32, _i32]
        L.bsfp8_dispatch_plan.restype = ctypes.c_int
        L.bsfp8_dispatch_plan.argtypes = [_vp, _vp, _i64, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp]
        L.bsfp8_dispatch.restype = ctypes.c_int
        L.bsfp8_dispatch.argtypes = [_vp, ctypes.c_int, _i64, _i64, _vp, _i32, _vp, _vp, _i64, _vp]
        L.bsfp8_dispatch_quantize.restype = ctypes.c_int
        L.bsfp8_dispatch_quantize.argtypes = [_vp, _i64, _i64, _vp, _i32, _vp, _i64, _vp, _i32, ctypes.c_int, ctypes.c_int,
                                              _vp, _vp, _vp, _vp, _vp, _vp]
        L.bsfp8_combine.restype = ctypes.c_int
        L.bsfp8_combine.argtypes = [_vp, ctypes.c_int, _i64, _i64, _vp, _i64, _i32, _vp, _vp, _vp, _vp]
        L.bsfp8_combine_grad.restype = ctypes.c_int
        L.bsfp8_combine_grad.argtypes = [_vp, ctypes.c_int, _i64, _i64, _vp, _i64, _vp, _i32, _vp, _vp, _vp, _vp]
        L.bsfp8_grouped_act_checkpoint.restype = ctypes.c_int
        L.bsfp8_grouped_act_checkpoint.argtypes = [ctypes.c_int, _vp, _vp, _i64, _i64, _vp, _i32, ctypes.c_int,
                                                   ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
        L.bsfp8_grouped_act_checkpoint_grad_workspace_bytes.restype = _sz
        L.bsfp8_grouped_act_checkpoint_grad_workspace_bytes.argtypes = [_i64, _i64]
        L.bsfp8_grouped_act_checkpoint_grad.restype = ctypes.c_int
        L.bsfp8_grouped_act_checkpoint_grad.argtypes = [ctypes.c_int, _vp, _vp, _vp, _vp, _i64, _i64, _vp, _i32,
                                                        ctypes.c_int, ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                                        _vp, _vp, _vp]
        L.bsfp8_strerror.restype = ctypes.c_char_p
        L.bsfp8_strerror.argtypes = [ctypes.c_int]
        _lib = L
    return _lib


def strerror(code):
    return lib().bsfp8_strerror(int(code)).decode()


def _check(rc, what):
    if rc != 0:
        raise BSFP8Error(f"{what}: {strerror(rc)} ({rc})")


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        return int(t)  # a raw address
    return t.data_ptr()


_U8 = (torch.uint8,)
_BF16 = (torch.bfloat16, torch.int16)  # bf16 data, or its bits viewed as int16
_F32 = (torch.float32,)
_I32 = (torch.int32,)
_F32_BITS = (torch.float32, torch.int32)
_STREAM = (torch.float32, torch.bfloat16)  # element types of a residual stream, parameters, gradients
_E4M3 = (torch.uint8, torch.float8_e4m3fn)


def _dev(t, what, dtypes):
    """Pointer of an argument that the kernels read or write: a contiguous device tensor of one
    of ``dtypes`` (checked in that order, so a wrong type is reported before a wrong device), a
    raw device address (int, not checked), or None.  A host tensor would hand the GPU a host
    pointer, and a tensor of another element type would be read with the wrong layout (an int64
    split_sizes tensor reads as sizes k_0, 0, k_1, 0, ...)."""
    if t is None or not isinstance(t, torch.Tensor):
        return _ptr(t)
    if t.dtype not in dtypes:
        raise TypeError(f"{what}: dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if not t.is_cuda:
        raise ValueError(f"{what}: a {t.device.type} tensor; the library takes device memory")
    if not t.is_contiguous():
        raise ValueError(f"{what}: not contiguous")
    return t.data_ptr()


def _quant(q, key, what, dtypes=_U8):
    return _dev(q.get(key), f"{what}[{key!r}]", dtypes)


def _need(t, nbytes, what):
    """A tensor argument must hold at least the bytes the kernels address for the given sizes and
    recipe (a buffer quantized with another recipe, or sized for other dims, would be read or
    written past its end); raw addresses are not checked."""
    if isinstance(t, torch.Tensor) and nbytes > 0 and t.numel() * t.element_size() < nbytes:
        raise ValueError(f"{what}: {t.numel() * t.element_size()} bytes, the call addresses {nbytes}")


def _need_quant(q, recipe, rows, cols, num_groups, which, what):
    """The quantized buffers of ``q`` against the layouts ``which`` of a [rows, cols] operand with
    ``num_groups`` groups: at least the size queries' bytes (alloc_quantized's sizes; a colwise
    buffer holds up to that bound, depending on the device split sizes).  With no rows nothing is
    addressed."""
    if rows == 0:
        return
    r = recipe & ~GEMM_FP8_MFMA
    if which & ROWWISE:
        _need(q.get("row_q"), rowwise_data_bytes(rows, cols, r), f"{what}['row_q']")
        _need(q.get("row_s"), rowwise_scale_bytes(rows, cols), f"{what}['row_s']")
    if which & COLWISE:
        _need(q.get("col_q"), colwise_data_bytes(rows, cols, num_groups, r), f"{what}['col_q']")
        _need(q.get("col_s"), colwise_scale_bytes(rows, cols, num_groups, r), f"{what}['col_s']")


def _col_s_types(recipe):
    return _F32 if (recipe & ~GEMM_FP8_MFMA) == RECIPE_PC else _U8


# torch's current stream as a raw handle, without building a Stream object for every call (a quarter of a
# small call's host time), where this torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None and _raw_device is not None and torch.cuda.is_initialized():
            return _raw_stream(_raw_device())
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _elsewhere(stream):
    """Whether a stream argument asks for another stream than the current one."""
    if stream is None or not torch.cuda.is_initialized():
        return False
    if isinstance(stream, torch.cuda.Stream):
        return stream != torch.cuda.current_stream()  # (also where only the device differs)
    return _stream(stream) != _stream(None)


def _on(stream):
    """The given stream (a torch stream or a raw handle) as the current one: what a call allocates itself
    then belongs to the stream that its kernels run on, and is not handed out again before they have run.
    Handle 0 is the default stream; ExternalStream would take it for no handle and make a stream of its own."""
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _load_native():
    """The checks, allocations and calls of the smallest launches in native code (csrc/binding.cpp), or None
    where it is not built: every call then goes through ctypes.  Loaded when first asked for, since it maps
    libbsfp8.so, which a process that only builds must not have done."""
    global _native
    try:
        _native = importlib.import_module("._native", __name__)
    except ImportError:
        _native = None
    return _native


def __getattr__(name):
    if name == "_native":
        return _load_native()
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


def _native_done(got, what):
    """Whether the native path took a call; raises for one that it made and that failed."""
    if got is None:
        return False
    if type(got) is int:
        _check(got, what)
    return True


def _use_native():
    if not torch.cuda.is_initialized():  # there are no device tensors
        return False
    return (_native if "_native" in globals() else _load_native()) is not None


# ------------------------------------------------------------------------------------------
# size queries
# ------------------------------------------------------------------------------------------

def colwise_rows_bound(capacity_rows, num_groups):
    return int(lib().bsfp8_colwise_rows_bound(capacity_rows, num_groups))


def colwise_data_bytes(capacity_rows, cols, num_groups, recipe=RECIPE_MX):
    return int(lib().bsfp8_colwise_data_bytes(capacity_rows, cols, num_groups, recipe))


def colwise_scale_bytes(capacity_rows, cols, num_groups, recipe):
    return int(lib().bsfp8_colwise_scale_bytes(capacity_rows, cols, num_groups, recipe))


def rowwise_data_bytes(rows, cols, recipe=RECIPE_MX):
    return int(lib().bsfp8_rowwise_data_bytes(rows, cols, recipe))


def rowwise_scale_bytes(rows, cols):
    return int(lib().bsfp8_rowwise_scale_bytes(rows, cols))


def alloc_quantized(capacity_rows, cols, num_groups, recipe, which, device="cuda"):
    """Output tensors for grouped_quantize, sized by the library's size queries.

    Returns a dict with row_q uint8 [R, C] (MXFP4: [R, C/2]), row_s uint8 [C/32, R], col_q uint8
    [bytes], col_s uint8 [bytes] (MX recipes) or float32 [bytes/4] (per-channel), for the
    requested layouts."""
    out = {}
    if which & ROWWISE:
        per = 2 if recipe == RECIPE_MX4 else 1
        out["row_q"] = torch.empty((capacity_rows, cols // per), dtype=torch.uint8, device=device)
        out["row_s"] = torch.empty((cols // 32, capacity_rows), dtype=torch.uint8, device=device)
    if which & COLWISE:
        out["col_q"] = torch.empty(colwise_data_bytes(capacity_rows, cols, num_groups, recipe), dtype=torch.uint8,
                                   device=device)
        nb = colwise_scale_bytes(capacity_rows, cols, num_groups, recipe)
        if recipe != RECIPE_PC:
            out["col_s"] = torch.empty(nb, dtype=torch.uint8, device=device)
        else:
            out["col_s"] = torch.empty(nb // 4, dtype=torch.float32, device=device)
    return out


# ------------------------------------------------------------------------------------------
# entry points
# ------------------------------------------------------------------------------------------

def grouped_quantize(x, split_sizes, recipe, which, out, zero_amax_scale=1e-30, status=None, stream=None,
                     capacity_rows=None, cols=None, noop_flag=None):
    """bsfp8_grouped_quantize on a bf16 [R, C] tensor; ``out`` holds the output tensors
    (see alloc_quantized), overwritten in place.  split_sizes: int32 device tensor, or None
    (rowwise, all rows live).  noop_flag: None, or a float32 device scalar; when it holds a
    nonzero value at run time the call leaves ``out`` (and ``status``) as they are."""
    if isinstance(x, torch.Tensor):
        R, C = x.shape if capacity_rows is None else (capacity_rows, cols)
    else:
        R, C = capacity_rows, cols
    E = 0 if split_sizes is None else int(split_sizes.numel())
    args = (_dev(x, "x", _BF16), R, C, _dev(split_sizes, "split_sizes", _I32), E, recipe, which,
            float(zero_amax_scale), _quant(out, "row_q", "out"), _quant(out, "row_s", "out"),
            _quant(out, "col_q", "out"), _quant(out, "col_s", "out", _col_s_types(recipe)),
            _dev(noop_flag, "noop_flag", _F32), _dev(status, "status", _I32), _stream(stream))
    _need(x, R * C * 2, "x")
    _need_quant(out, recipe, R, C, max(E, 1), which, "out")
    rc = lib().bsfp8_grouped_quantize(*args)
    _check(rc, "grouped_quantize")
    return out


def grouped_act_quantize(activation, h, split_sizes, recipe, which, out, probs=None, dy=None, status=None,
                         stream=None):
    """bsfp8_grouped_act_quantize: the scaled squared ReLU (ACT_SRELU) of the bf16 [R, C] tensor
    h, or its gradient (ACT_SRELU_GRAD, with the bf16 gradient dy [R, C]); or the scaled SwiGLU
    (ACT_SWIGLU) of h = (a | b) [R, 2F], or its gradient (ACT_SWIGLU_GRAD, dy [R, F]); times the
    float32 per-row probs (None: 1), quantized into ``out`` with an MX recipe.  ``out`` comes
    from alloc_quantized for [R, C], [R, F] (ACT_SWIGLU) or [R, 2F] (ACT_SWIGLU_GRAD)."""
    R, C = h.shape
    if activation in (ACT_SWIGLU, ACT_SWIGLU_GRAD):
        if C % 2:
            raise ValueError("grouped_act_quantize: a GLU input has an even number of columns")
        C //= 2
    E = int(split_sizes.numel())
    args = (activation, _dev(h, "h", _BF16), _dev(probs, "probs", _F32), _dev(dy, "dy", _BF16), R, C,
            _dev(split_sizes, "split_sizes", _I32), E, recipe, which, _quant(out, "row_q", "out"),
            _quant(out, "row_s", "out"), _quant(out, "col_q", "out"), _quant(out, "col_s", "out"),
            _dev(status, "status", _I32), _stream(stream))
    _need_quant(out, recipe, R, 2 * C if activation == ACT_SWIGLU_GRAD else C, E, which, "out")
    rc = lib().bsfp8_grouped_act_quantize(*args)
    _check(rc, "grouped_act_quantize")
    return out


def grouped_gemm_wgrad(dy_q, n, x_q, h, split_sizes, capacity_rows, recipe, out, accumulate=False, status=None,
                       stream=None):
    """bsfp8_grouped_gemm_wgrad: dy_q / x_q are the colwise dicts of grouped_quantize; out is
    fp32 [E, n, h] (overwritten, or accumulated into with ``accumulate``).  recipe: the data
    recipe, or RECIPE_MX | GEMM_FP8_MFMA for the MXFP8 operands on the scaled fp8 MFMA."""
    E = int(split_sizes.numel())
    cs = _col_s_types(recipe)
    args = (_quant(dy_q, "col_q", "dy_q"), _quant(dy_q, "col_s", "dy_q", cs), n, _quant(x_q, "col_q", "x_q"),
            _quant(x_q, "col_s", "x_q", cs), h, _dev(split_sizes, "split_sizes", _I32), E, capacity_rows, recipe,
            _dev(out, "out", _F32_BITS), 1 if accumulate else 0, _dev(status, "status", _I32), _stream(stream))
    _need_quant(dy_q, recipe, capacity_rows, n, E, COLWISE, "dy_q")
    _need_quant(x_q, recipe, capacity_rows, h, E, COLWISE, "x_q")
    _need(out, E * n * h * 4, "out")
    rc = lib().bsfp8_grouped_gemm_wgrad(*args)
    _check(rc, "grouped_gemm_wgrad")
    return out


def grouped_gemm_fprop(x_q, k, w_q, n, split_sizes, capacity_rows, out, out_dtype=OUT_F32, status=None,
                       stream=None, recipe=RECIPE_MX):
    """bsfp8_grouped_gemm_fprop: x_q is the rowwise dict of x [R, k], w_q the rowwise dict of the
    weight [E*n, k], both of ``recipe`` (MX or MX4; RECIPE_MX | GEMM_FP8_MFMA multiplies MX
    operands on the scaled fp8 MFMA); out is [R, n] fp32 or bf16 (rows past
    sum(split_sizes) untouched)."""
    E = int(split_sizes.numel())
    args = (_quant(x_q, "row_q", "x_q"), _quant(x_q, "row_s", "x_q"), capacity_rows, k, _quant(w_q, "row_q", "w_q"),
            _quant(w_q, "row_s", "w_q"), n, _dev(split_sizes, "split_sizes", _I32), E, recipe,
            _dev(out, "out", _F32_BITS if out_dtype == OUT_F32 else _BF16), out_dtype,
            _dev(status, "status", _I32), _stream(stream))
    _need_quant(x_q, recipe, capacity_rows, k, E, ROWWISE, "x_q")
    _need_quant(w_q, recipe, E * n, k, 1, ROWWISE, "w_q")
    _need(out, capacity_rows * n * (4 if out_dtype == OUT_F32 else 2), "out")
    rc = lib().bsfp8_grouped_gemm_fprop(*args)
    _check(rc, "grouped_gemm_fprop")
    return out


def grouped_gemm_dgrad(dy_q, n, w_q, k, split_sizes, capacity_rows, out, out_dtype=OUT_F32, status=None,
                       stream=None, recipe=RECIPE_MX):
    """bsfp8_grouped_gemm_dgrad: dy_q is the rowwise dict of dy [R, n]; w_q the colwise dict of the
    weight viewed as [E*n, k] quantized with split sizes [n] * E (blocks of 32 along n inside each
    expert); out is [R, k] fp32 or bf16: out[off_e + t] = dy[off_e + t] @ W_e (rows past
    sum(split_sizes) untouched)."""
    E = int(split_sizes.numel())
    args = (_quant(dy_q, "row_q", "dy_q"), _quant(dy_q, "row_s", "dy_q"), capacity_rows, n,
            _quant(w_q, "col_q", "w_q"), _quant(w_q, "col_s", "w_q"), k, _dev(split_sizes, "split_sizes", _I32), E,
            recipe, _dev(out, "out", _F32_BITS if out_dtype == OUT_F32 else _BF16), out_dtype,
            _dev(status, "status", _I32), _stream(stream))
    _need_quant(dy_q, recipe, capacity_rows, n, E, ROWWISE, "dy_q")
    # the weight [E*n, k] quantized colwise with split sizes n: E groups of 128 * ceil(n / 128) rows
    np_ = 128 * ((n + 127) // 128)
    per = 2 if (recipe & ~GEMM_FP8_MFMA) == RECIPE_MX4 else 1
    _need(w_q.get("col_q"), k * E * np_ // per, "w_q['col_q']")
    _need(w_q.get("col_s"), k * E * np_ // 32, "w_q['col_s']")
    _need(out, capacity_rows * k * (4 if out_dtype == OUT_F32 else 2), "out")
    rc = lib().bsfp8_grouped_gemm_dgrad(*args)
    _check(rc, "grouped_gemm_dgrad")
    return out


# ------------------------------------------------------------------------------------------
# gated feed-forward projection
# ------------------------------------------------------------------------------------------

def _buf(t, what, key, dtypes, nbytes):
    """_dev and _need in one, the argument's name put together only for an error."""
    if t is None or not isinstance(t, torch.Tensor):
        return _ptr(t)
    if t.dtype not in dtypes or not t.is_cuda or not t.is_contiguous():
        return _dev(t, what if key is None else f"{what}[{key!r}]", dtypes)
    if t.numel() * t.element_size() < nbytes:
        _need(t, nbytes, what if key is None else f"{what}[{key!r}]")
    return t.data_ptr()


def _glu_quantized(q, rows, cols, num_groups):
    """What a dict of quantized outputs [rows, cols] asks for: the layouts and the four pointers."""
    if not q:
        return 0, None, None, None, None
    which, ptrs = 0, [None] * 4
    if q.get("row_q") is not None:
        which |= ROWWISE
        ptrs[0] = _buf(q["row_q"], "out", "row_q", _U8, rows * cols)
        ptrs[1] = _buf(q.get("row_s"), "out", "row_s", _U8, rows * cols // 32)
    if q.get("col_q") is not None:
        which |= COLWISE
        bound = 128 * ((rows + 127 * num_groups) // 128) if rows else 0
        ptrs[2] = _buf(q["col_q"], "out", "col_q", _U8, cols * bound)
        ptrs[3] = _buf(q.get("col_s"), "out", "col_s", _U8, cols * bound // 32)
    return (which, *ptrs)


def _glu_result(q, **more):
    out = {k: v for k, v in more.items() if v is not None}
    if q:
        out.update(q)
    return out


def grouped_gemm_swiglu(x_q, hidden, w_q, ffn, split_sizes, capacity_rows, recipe=RECIPE_MX, probs=None, ab=None,
                        y=None, y_dtype=OUT_BF16, out=None, status=None, stream=None):
    """bsfp8_grouped_gemm_swiglu: y = probs * silu(a) * b with (a | b) = x W1_e^T in one kernel.  x_q is the
    rowwise dict of x [R, hidden], w_q the rowwise dict of W1 [E * 2 ffn, hidden] (each expert's a rows,
    then its b rows).  Any of: ab bf16 [R, 2 ffn] (kept for the gradient), y [R, ffn] (bf16 or fp32, as
    y_dtype says), out (alloc_quantized for [R, ffn]) receives y quantized in the layouts it holds.
    Returns a dict of those.  Rows past sum(split_sizes) are untouched."""
    q = out or {}
    if _use_native() and _native_done(_native.swiglu(
            x_q.get("row_q"), x_q.get("row_s"), capacity_rows, hidden, w_q.get("row_q"), w_q.get("row_s"), ffn, split_sizes,
            recipe, y_dtype, probs, ab, y, q.get("row_q"), q.get("row_s"), q.get("col_q"), q.get("col_s"), status,
            _stream(stream)), "grouped_gemm_swiglu"):
        return _glu_result(out, ab=ab, y=y)
    E, R = int(split_sizes.numel()), capacity_rows
    f32 = y_dtype == OUT_F32
    which, *q = _glu_quantized(out, R, ffn, E)
    rc = lib().bsfp8_grouped_gemm_swiglu(
        _buf(x_q.get("row_q"), "x_q", "row_q", _U8, R * hidden),
        _buf(x_q.get("row_s"), "x_q", "row_s", _U8, R * hidden // 32), R, hidden,
        _buf(w_q.get("row_q"), "w_q", "row_q", _U8, E * 2 * ffn * hidden),
        _buf(w_q.get("row_s"), "w_q", "row_s", _U8, E * 2 * ffn * hidden // 32), ffn,
        _buf(probs, "probs", None, _F32, R * 4), _dev(split_sizes, "split_sizes", _I32), E, recipe,
        _buf(ab, "ab", None, _BF16, R * ffn * 4),
        _buf(y, "y", None, _F32_BITS if f32 else _BF16, R * ffn * (4 if f32 else 2)), y_dtype, which, *q,
        _dev(status, "status", _I32), _stream(stream))
    if rc:
        _check(rc, "grouped_gemm_swiglu")
    return _glu_result(out, ab=ab, y=y)


def grouped_gemm_swiglu_grad_workspace_bytes(capacity_rows, ffn, num_groups):
    return int(lib().bsfp8_grouped_gemm_swiglu_grad_workspace_bytes(capacity_rows, ffn, num_groups))


def grouped_gemm_swiglu_grad(dy_q, hidden, w_q, ffn, ab, split_sizes, capacity_rows, recipe=RECIPE_MX, probs=None,
                             dab=None, out=None, dprobs=None, workspace=None, status=None, stream=None):
    """bsfp8_grouped_gemm_swiglu_grad: from the gradient at the second projection's output, dy_q (the
    rowwise dict of dy [R, hidden]), that projection's weight w_q (the colwise dict of W2 viewed as
    [E * hidden, ffn] with split sizes [hidden] * E) and the forward's ab, the gradient (da | db), as
    bf16 dab [R, 2 ffn] and / or quantized into out (alloc_quantized for [R, 2 ffn]), and that of the
    probabilities, dprobs fp32 [R].  Returns a dict of those.  workspace: a device tensor of
    grouped_gemm_swiglu_grad_workspace_bytes, for dprobs (None: a new one)."""
    if dprobs is not None and workspace is None and _elsewhere(stream):
        with _on(stream):
            return grouped_gemm_swiglu_grad(dy_q, hidden, w_q, ffn, ab, split_sizes, capacity_rows, recipe, probs, dab, out,
                                            dprobs, None, status)
    q = out or {}
    if _use_native() and _native_done(_native.swiglu_grad(
            dy_q.get("row_q"), dy_q.get("row_s"), capacity_rows, hidden, w_q.get("col_q"), w_q.get("col_s"), ffn,
            split_sizes, recipe, ab, probs, dab, q.get("row_q"), q.get("row_s"), q.get("col_q"), q.get("col_s"), dprobs,
            workspace, status, _stream(stream)), "grouped_gemm_swiglu_grad"):
        return _glu_result(out, dab=dab, dprobs=dprobs)
    E, R = int(split_sizes.numel()), capacity_rows
    which, *q = _glu_quantized(out, R, 2 * ffn, E)
    hp = 128 * ((hidden + 127) // 128)
    ptrs = (_buf(dy_q.get("row_q"), "dy_q", "row_q", _U8, R * hidden),
            _buf(dy_q.get("row_s"), "dy_q", "row_s", _U8, R * hidden // 32), R, hidden,
            _buf(w_q.get("col_q"), "w_q", "col_q", _U8, ffn * E * hp),
            _buf(w_q.get("col_s"), "w_q", "col_s", _U8, ffn * E * hp // 32), ffn,
            _buf(ab, "ab", None, _BF16, R * ffn * 4), _buf(probs, "probs", None, _F32, R * 4),
            _dev(split_sizes, "split_sizes", _I32), E, recipe, _buf(dab, "dab", None, _BF16, R * ffn * 4))
    pws = None
    if dprobs is not None:
        need = grouped_gemm_swiglu_grad_workspace_bytes(R, ffn, E)
        if workspace is None and need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=split_sizes.device)
        if workspace is not None:
            pws = _buf(workspace, "workspace", None, (workspace.dtype,), need)
    rc = lib().bsfp8_grouped_gemm_swiglu_grad(*ptrs, which, *q, _buf(dprobs, "dprobs", None, _F32, R * 4), pws,
                                              _dev(status, "status", _I32), _stream(stream))
    if rc:
        _check(rc, "grouped_gemm_swiglu_grad")
    return _glu_result(out, dab=dab, dprobs=dprobs)


# ------------------------------------------------------------------------------------------
# norms around a block
# ------------------------------------------------------------------------------------------

def _dtype_code(t):
    return F32 if t.dtype == torch.float32 else BF16


def _like(t, shape, what, dtype=None):
    """A tensor argument of exactly this shape (and element type, where given)."""
    if t is None:
        return
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {None if shape is None else tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what}: dtype {t.dtype}, expected {dtype}")


def _out(t, shape, what, dtypes):
    """Pointer of an output tensor that the caller gave, of this shape and one of these types, or None."""
    if t is None:
        return None
    p = _dev(t, what, dtypes)
    _like(t, shape, what)
    return p


def _check_norm_block(shape, y, post_weight, pre_weight, gate, gate_kind):
    rows, cols = shape
    _like(y, shape, "y")
    _like(post_weight, (cols,), "post_weight")
    _like(pre_weight, (cols,), "pre_weight")
    if gate_kind == GATE_CHANNEL:
        _like(gate, (cols,), "gate")
    elif gate_kind == GATE_TOKEN:
        _like(gate, (rows,), "gate")


def residual_norm(x, y=None, post_weight=None, pre_weight=None, gate=None, gate_kind=GATE_NONE, x_scale=1.0,
                  y_scale=1.0, eps=1e-6, weight_offset=0.0, r=None, n=None, rstd_y=None, rstd_r=None, stream=None):
    """bsfp8_residual_norm on the residual stream x [rows, cols] (fp32 or bf16) and the block's
    output y [rows, cols] (bf16):

        r = x_scale * x + y_scale * gate * (y * rstd_y * (post_weight + weight_offset))
        n = r * rstd_r * (pre_weight + weight_offset)

    post_weight, pre_weight: fp32 [cols]; None leaves out that norm (without pre_weight there is no
    n).  gate: fp32 [cols] (GATE_CHANNEL) or [rows] (GATE_TOKEN).  Returns a dict of r (x's type), n
    (bf16), rstd_y and rstd_r (fp32 [rows], for the gradient), in the tensors given or in new ones;
    r may be x.  Data begins at multiples of 16 bytes."""
    if _elsewhere(stream):
        with _on(stream):
            return residual_norm(x, y, post_weight, pre_weight, gate, gate_kind, x_scale, y_scale, eps, weight_offset, r, n,
                                 rstd_y, rstd_r)
    if _use_native():
        got = _native.residual_norm(x, y, post_weight, pre_weight, gate, gate_kind, x_scale, y_scale, eps, weight_offset,
                                    r, n, rstd_y, rstd_r, _stream(stream))
        if _native_done(got, "residual_norm"):
            out = {"r": got[0]}
            if pre_weight is not None:
                out["n"], out["rstd_r"] = got[1], got[3]
            if post_weight is not None:
                out["rstd_y"] = got[2]
            return out
    if x.dim() != 2:
        raise ValueError("residual_norm: x is [rows, cols]")
    shape = rows, cols = x.shape
    px = _dev(x, "x", _STREAM)
    py, pw, qw = _dev(y, "y", _BF16), _dev(post_weight, "post_weight", _F32), _dev(pre_weight, "pre_weight", _F32)
    pg = _dev(gate, "gate", _F32)
    _check_norm_block(shape, y, post_weight, pre_weight, gate, gate_kind)
    # given tensors are checked, new ones are as they have to be
    out, pn, prr, pry = {}, None, None, None
    if r is None:
        out["r"] = r = torch.empty_like(x)
        pr = r.data_ptr()
    else:
        out["r"], pr = r, _out(r, shape, "r", (x.dtype,))
    if pre_weight is not None:
        if n is None:
            n = torch.empty_like(x, dtype=torch.bfloat16)
            pn = n.data_ptr()
        else:
            pn = _out(n, shape, "n", _BF16)
        out["n"] = n
        if rstd_r is None:
            rstd_r = x.new_empty(rows, dtype=torch.float32)
            prr = rstd_r.data_ptr()
        else:
            prr = _out(rstd_r, (rows,), "rstd_r", _F32)
        out["rstd_r"] = rstd_r
    else:
        pn, prr = _out(n, shape, "n", _BF16), _out(rstd_r, (rows,), "rstd_r", _F32)
    if post_weight is not None:
        if rstd_y is None:
            rstd_y = x.new_empty(rows, dtype=torch.float32)
            pry = rstd_y.data_ptr()
        else:
            pry = _out(rstd_y, (rows,), "rstd_y", _F32)
        out["rstd_y"] = rstd_y
    else:
        pry = _out(rstd_y, (rows,), "rstd_y", _F32)
    rc = lib().bsfp8_residual_norm(rows, cols, px, F32 if x.dtype is torch.float32 else BF16, py, pw, qw, pg, gate_kind,
                                   x_scale, y_scale, eps, weight_offset, pr, pn, pry, prr, _stream(stream))
    if rc:
        _check(rc, "residual_norm")
    return out


def residual_norm_grad_workspace_bytes(rows, cols):
    return int(lib().bsfp8_residual_norm_grad_workspace_bytes(rows, cols))


def residual_norm_grad(dn, dr, r=None, rstd_r=None, pre_weight=None, y=None, rstd_y=None, post_weight=None, gate=None,
                       gate_kind=GATE_NONE, x_scale=1.0, y_scale=1.0, weight_offset=0.0, dx=None, dy=None,
                       dpre_weight=None, dpost_weight=None, dgate=None, accumulate=False, workspace=None, stream=None):
    """bsfp8_residual_norm_grad: the gradient of residual_norm from dn [rows, cols] (bf16, the gradient
    at n, or None) and dr [rows, cols] (the stream's type, the gradient at r, or None), with r, rstd_r,
    rstd_y as the forward returned them.  Returns a dict of dx (the stream's type), dy (bf16) and, for
    the weights and the gate that are there, dpre_weight, dpost_weight, dgate (fp32), in the tensors
    given or in new ones.  accumulate: the weights' and a channel gate's gradients are added to the
    tensors given."""
    if _elsewhere(stream):
        with _on(stream):
            return residual_norm_grad(dn, dr, r, rstd_r, pre_weight, y, rstd_y, post_weight, gate, gate_kind, x_scale,
                                      y_scale, weight_offset, dx, dy, dpre_weight, dpost_weight, dgate, accumulate,
                                      workspace)
    if _use_native():
        got = _native.residual_norm_grad(dn, dr, r, rstd_r, pre_weight, y, rstd_y, post_weight, gate, gate_kind, x_scale,
                                         y_scale, weight_offset, dx, dy, dpre_weight, dpost_weight, dgate, accumulate,
                                         workspace, _stream(stream))
        if _native_done(got, "residual_norm_grad"):
            out = {"dx": got[0]}
            for name, of, value in (("dy", y, got[1]), ("dpre_weight", pre_weight, got[2]),
                                    ("dpost_weight", post_weight, got[3]), ("dgate", gate, got[4])):
                if of is not None:
                    out[name] = value
            return out
    ref = dr if dr is not None else r
    if ref is None:
        raise ValueError("residual_norm_grad: neither dr nor (dn and r)")
    if ref.dim() != 2:
        raise ValueError("residual_norm_grad: r and dr are [rows, cols]")
    shape = rows, cols = ref.shape
    dtype = ref.dtype
    args = (F32 if dtype is torch.float32 else BF16, _dev(dn, "dn", _BF16), _dev(dr, "dr", _STREAM),
            _dev(r, "r", _STREAM), _dev(rstd_r, "rstd_r", _F32), _dev(pre_weight, "pre_weight", _F32),
            _dev(y, "y", _BF16), _dev(rstd_y, "rstd_y", _F32), _dev(post_weight, "post_weight", _F32),
            _dev(gate, "gate", _F32))
    _like(dn, shape, "dn")
    _like(dr, shape, "dr", dtype)
    _like(r, shape, "r", dtype)
    _like(rstd_r, (rows,), "rstd_r")
    _like(rstd_y, (rows,), "rstd_y")
    _check_norm_block(shape, y, post_weight, pre_weight, gate, gate_kind)
    if accumulate and any(w is not None and d is None for w, d in (
            (pre_weight, dpre_weight), (post_weight, dpost_weight),
            (gate if gate_kind == GATE_CHANNEL else None, dgate))):
        raise ValueError("residual_norm_grad: accumulate needs the gradients to add to")
    out = {}

    def put(name, given, like, out_shape, dtypes):
        # the pointer of an output: the tensor given, or a new one where the call has what it is the gradient of
        if given is None:
            if like is None:
                return None
            given = torch.empty_like(like)
            out[name] = given
            return given.data_ptr()
        if like is not None:
            out[name] = given
        return _out(given, out_shape, name, dtypes)

    pdx = put("dx", dx, ref, shape, (dtype,))
    pdy = put("dy", dy, y, shape, _BF16)
    pre = put("dpre_weight", dpre_weight, pre_weight, (cols,), _F32)
    post = put("dpost_weight", dpost_weight, post_weight, (cols,), _F32)
    pgate = put("dgate", dgate, gate, None if gate is None else gate.shape, _F32)
    need = residual_norm_grad_workspace_bytes(rows, cols)
    if workspace is None:
        workspace = ref.new_empty(need, dtype=torch.uint8)
    else:
        _need(workspace, need, "workspace")
    rc = lib().bsfp8_residual_norm_grad(
        rows, cols, *args, gate_kind, x_scale, y_scale, weight_offset, pdx, pdy, pre, post, pgate,
        1 if accumulate else 0, _dev(workspace, "workspace", (workspace.dtype,)), _stream(stream))
    if rc:
        _check(rc, "residual_norm_grad")
    return out


# ------------------------------------------------------------------------------------------
# AdamW
# ------------------------------------------------------------------------------------------

class _AdamTensor(ctypes.Structure):
    _fields_ = [("param", _vp), ("grad", _vp), ("exp_avg", _vp), ("exp_avg_sq", _vp), ("exp_avg_scale", _vp),
                ("exp_avg_sq_scale", _vp), ("copy", _vp), ("numel", _i64), ("lr_scale", ctypes.c_float),
                ("decay_scale", ctypes.c_float)]


class AdamWPlan:
    """The tensors of an AdamW step, their addresses laid out on the device once (adamw_plan).  It holds
    the tensors; they stay where they are as long as it is used."""

    def __init__(self, table, num_tensors, num_chunks, param_dtype, grad_dtype, state, tensors):
        self.table, self.num_tensors, self.num_chunks = table, num_tensors, num_chunks
        self.param_dtype, self.grad_dtype, self.state, self.tensors = param_dtype, grad_dtype, state, tensors


def adamw_plan(params, grads, exp_avgs, exp_avg_sqs, exp_avg_scales=None, exp_avg_sq_scales=None, copies=None,
               lr_scales=None, decay_scales=None):
    """Plan of an AdamW step over lists of tensors: params and grads (fp32 or bf16, one type each),
    states exp_avgs and exp_avg_sqs as fp32, or as e4m3 codes (uint8 or float8_e4m3fn) with the fp32
    scales [ceil(numel / 128)] in exp_avg_scales and exp_avg_sq_scales (the second state is sqrt(v);
    zeroed codes and scales are a valid start).  copies: bf16 tensors (or None) that receive the new
    params.  lr_scales, decay_scales: factors on lr and weight_decay per tensor (default 1).  Laid out once
    for tensors that stay where they are: it takes some 4 us per tensor on the host."""
    n = len(params)
    if n == 0:
        raise ValueError("adamw_plan: no tensors")
    q8 = exp_avg_scales is not None
    if q8 != (exp_avg_sq_scales is not None):
        raise ValueError("adamw_plan: exp_avg_scales and exp_avg_sq_scales come together")
    none = [None] * n
    lists = dict(grads=grads, exp_avgs=exp_avgs, exp_avg_sqs=exp_avg_sqs, exp_avg_scales=exp_avg_scales or none,
                 exp_avg_sq_scales=exp_avg_sq_scales or none, copies=copies or none, lr_scales=lr_scales or [1.0] * n,
                 decay_scales=decay_scales or [1.0] * n)
    for name, v in lists.items():
        if len(v) != n:
            raise ValueError(f"adamw_plan: {len(v)} {name} for {n} params")
    ptypes, gtypes = (params[0].dtype,), (grads[0].dtype,)
    for name, t in (("params", ptypes), ("grads", gtypes)):
        if t[0] not in _STREAM:
            raise TypeError(f"{name}[0]: dtype {t[0]}, expected torch.float32 or torch.bfloat16")
    stypes = _E4M3 if q8 else _F32
    device = params[0].device
    table, numels = (_AdamTensor * n)(), (_i64 * n)()
    for i, (p, g, m, v, ms, vs, c, ls, ds) in enumerate(zip(params, *lists.values())):
        size = p.numel()
        for what, t, types, count in (("params", p, ptypes, size), ("grads", g, gtypes, size),
                                      ("exp_avgs", m, stypes, size), ("exp_avg_sqs", v, stypes, size),
                                      ("exp_avg_scales", ms, _F32, (size + 127) // 128),
                                      ("exp_avg_sq_scales", vs, _F32, (size + 127) // 128),
                                      ("copies", c, (torch.bfloat16,), size)):
            if t is None:
                continue
            _dev(t, f"{what}[{i}]", types)
            if t.numel() != count:
                raise ValueError(f"{what}[{i}]: {t.numel()} elements, expected {count}")
            if t.device != device:
                raise ValueError(f"{what}[{i}]: on {t.device}, params[0] on {device}")
        numels[i] = size
        table[i] = _AdamTensor(p.data_ptr(), g.data_ptr(), m.data_ptr(), v.data_ptr(), _ptr(ms), _ptr(vs), _ptr(c),
                               size, ls, ds)
    chunks = _i64()
    nbytes = lib().bsfp8_adamw_plan_bytes(numels, n, ctypes.byref(chunks))
    host = torch.empty(max(1, nbytes), dtype=torch.uint8)
    pd, gd, st = _dtype_code(params[0]), _dtype_code(grads[0]), STATE_8BIT if q8 else STATE_F32
    _check(lib().bsfp8_adamw_plan(table, n, pd, gd, st, host.data_ptr(), nbytes), "adamw_plan")
    kept = (list(params),) + tuple(lists.values())[:6]
    return AdamWPlan(host.to(device), n, chunks.value, pd, gd, st, kept)


def adamw_step(plan, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1, lr_dev=None, step_dev=None,
               grad_scale=None, noop_flag=None, stream=None, seed=None):
    """bsfp8_adamw_step: one AdamW step over the plan's tensors, in place.  step counts from 1.  Device
    scalars: lr_dev (fp32) and step_dev (int32) replace lr and step (for a captured graph), grad_scale
    (fp32) multiplies the gradients, a nonzero noop_flag (fp32) leaves everything as it is.

    seed: an int, with 8-bit states, rounds them stochastically (bsfp8_adamw_step_stochastic; the same seed and
    step give the same states).  Train with one: rounded to nearest (None, with a warning), an element's states
    stop following its gradients where another element holds its block's scale."""
    args = (plan.table.data_ptr(), plan.num_tensors, plan.num_chunks, plan.param_dtype, plan.grad_dtype, plan.state, lr,
            beta1, beta2, eps, weight_decay, step, _dev(lr_dev, "lr_dev", _F32), _dev(step_dev, "step_dev", _I32),
            _dev(grad_scale, "grad_scale", _F32), _dev(noop_flag, "noop_flag", _F32))
    if seed is None:
        if plan.state == STATE_8BIT:
            warnings.warn("adamw_step: 8-bit states rounded to nearest do not follow changes of less than half a code's step "
                          "(3 to 6%) a step; give a seed to train with them", stacklevel=2)
        _check(lib().bsfp8_adamw_step(*args, _stream(stream)), "adamw_step")
    else:
        _check(lib().bsfp8_adamw_step_stochastic(*args, int(seed) & 0xFFFFFFFFFFFFFFFF, _stream(stream)), "adamw_step")


# ------------------------------------------------------------------------------------------
# tokens to their experts and back
# ------------------------------------------------------------------------------------------

def _arg(t, what, dtypes, shape=None):
    """Pointer of a tensor argument of the calls below: as _dev checks it, on the current device, of this shape."""
    p = _dev(t, what, dtypes)
    if isinstance(t, torch.Tensor):
        if shape is not None:
            _like(t, shape, what)
        if t.get_device() != torch.cuda.current_device():
            raise ValueError(f"{what}: on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    return p


def _layout(q, key, what):
    """Pointer of one of a dict's quantized buffers, or of none."""
    return _arg(q.get(key), f"{what}[{key!r}]", _U8)


def _here():
    """What the native calls below begin with: the current device and its stream."""
    if _raw_device is None:
        return torch.cuda.current_device(), _stream(None)
    return _raw_device(), _stream(None)


def _matrix(t, what, dtypes):
    """Pointer and shape of a [rows, cols] tensor, which has to be given."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{what}: a two-dimensional tensor is needed")
    return _arg(t, what, dtypes), t.shape


def _workspace(workspace, nbytes, like):
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device) if nbytes > 0 else None
    _need(workspace, nbytes, "workspace")
    _arg(workspace, "workspace", (workspace.dtype,))
    return workspace


def route_topk_workspace_bytes(tokens, num_experts):
    return int(lib().bsfp8_route_topk_workspace_bytes(tokens, num_experts))


def route_topk(logits, top_k, scoring=ROUTE_SOFTMAX, bias=None, renormalize=True, scale=1.0, probs=None, experts=None,
               score_sum=None, workspace=None, stream=None):
    """bsfp8_route_topk: each token's top_k experts and their probabilities from the router's logits [tokens, experts]
    (fp32 or bf16).  scoring: ROUTE_SOFTMAX or ROUTE_SIGMOID; bias: fp32 [experts], moves the choice alone; renormalize:
    the chosen scores are divided by their sum; then they are multiplied by scale.  A logit of -inf masks an expert.
    score_sum: fp32 [experts], receives the sum of the scores over the tokens (for a load-balancing loss).  Returns a
    dict of probs (fp32 [tokens, top_k]), experts (int32, -1 where none is left) and score_sum, where given."""
    if _elsewhere(stream):
        with _on(stream):
            return route_topk(logits, top_k, scoring, bias, renormalize, scale, probs, experts, score_sum, workspace)
    if _use_native():
        got = _native.route_topk(*_here(), logits, top_k, scoring, bias, renormalize, scale, probs, experts, score_sum,
                                 workspace)
        if _native_done(got, "route_topk"):
            out = {"probs": got[0], "experts": got[1]}
            if score_sum is not None:
                out["score_sum"] = score_sum
            return out
    pl, (T, E) = _matrix(logits, "logits", _STREAM)
    pb, ps = _arg(bias, "bias", _F32, (E,)), _arg(score_sum, "score_sum", _F32, (E,))
    if probs is None:
        probs = logits.new_empty((T, top_k), dtype=torch.float32)
    if experts is None:
        experts = logits.new_empty((T, top_k), dtype=torch.int32)
    pp, pe = _arg(probs, "probs", _F32, (T, top_k)), _arg(experts, "experts", _I32, (T, top_k))
    if score_sum is not None:
        workspace = _workspace(workspace, route_topk_workspace_bytes(T, E), logits)
    rc = lib().bsfp8_route_topk(pl, _dtype_code(logits), T, E, top_k, scoring, pb, 1 if renormalize else 0, scale, pp, pe,
                                ps, _ptr(workspace) if score_sum is not None else None, _stream(stream))
    _check(rc, "route_topk")
    out = {"probs": probs, "experts": experts}
    if score_sum is not None:
        out["score_sum"] = score_sum
    return out


def route_topk_grad(dprobs, logits, experts, scoring=ROUTE_SOFTMAX, renormalize=True, scale=1.0, dscore_sum=None,
                    dlogits=None, stream=None):
    """bsfp8_route_topk_grad: the gradient at the logits, of their type, from dprobs (fp32 [tokens, top_k]), dscore_sum
    (fp32 [experts] or None), and the experts that route_topk chose."""
    if _elsewhere(stream):
        with _on(stream):
            return route_topk_grad(dprobs, logits, experts, scoring, renormalize, scale, dscore_sum, dlogits)
    if _use_native():
        got = _native.route_topk_grad(*_here(), dprobs, logits, experts, scoring, renormalize, scale, dscore_sum, dlogits)
        if _native_done(got, "route_topk_grad"):
            return got[0]
    pl, (T, E) = _matrix(logits, "logits", _STREAM)
    pe, (_, K) = _matrix(experts, "experts", _I32)
    _like(experts, (T, K), "experts")
    pp, ps = _arg(dprobs, "dprobs", _F32, (T, K)), _arg(dscore_sum, "dscore_sum", _F32, (E,))
    if dlogits is None:
        dlogits = torch.empty_like(logits)
    pd = _arg(dlogits, "dlogits", (logits.dtype,), (T, E))
    rc = lib().bsfp8_route_topk_grad(pp, pl, _dtype_code(logits), pe, T, E, K, scoring, 1 if renormalize else 0, scale, ps,
                                     pd, _stream(stream))
    _check(rc, "route_topk_grad")
    return dlogits


def dispatch_plan_workspace_bytes(tokens, top_k, num_experts):
    return int(lib().bsfp8_dispatch_plan_workspace_bytes(tokens, top_k, num_experts))


def dispatch_plan(experts, num_experts, probs=None, out=None, workspace=None, stream=None):
    """bsfp8_dispatch_plan: the choices of experts (int32 [tokens, top_k]; one outside [0, num_experts) is dropped) sorted
    by expert.  Returns a dict of splits (int32 [num_experts], the split_sizes of the grouped calls), rows (int32
    [tokens, top_k], each choice's row or -1), choices (int32 [tokens * top_k], each row's choice or -1 past the last)
    and, with probs (fp32 [tokens, top_k]), probs (fp32 [tokens * top_k], each row's, 0 past the last), in the tensors of
    ``out`` or in new ones."""
    if _elsewhere(stream):
        with _on(stream):
            return dispatch_plan(experts, num_experts, probs, out, workspace)
    given = out or {}
    if _use_native():
        got = _native.dispatch_plan(*_here(), experts, num_experts, probs, given.get("splits"), given.get("rows"),
                                    given.get("choices"), None if probs is None else given.get("probs"), workspace)
        if _native_done(got, "dispatch_plan"):
            out = {"splits": got[0], "rows": got[1], "choices": got[2]}
            if probs is not None:
                out["probs"] = got[3]
            return out
    pe, (T, K) = _matrix(experts, "experts", _I32)
    pp, N = _arg(probs, "probs", _F32, (T, K)), T * K
    ptrs, out = [], {}
    for name, shape, dtype in (("splits", (num_experts,), torch.int32), ("rows", (T, K), torch.int32),
                               ("choices", (N,), torch.int32), ("probs", (N,), torch.float32)):
        if name == "probs" and probs is None:
            ptrs.append(None)
            continue
        t = given.get(name)
        if t is None:
            t = experts.new_empty(shape, dtype=dtype)
        ptrs.append(_arg(t, f"out[{name!r}]", (dtype,), shape))
        out[name] = t
    workspace = _workspace(workspace, dispatch_plan_workspace_bytes(T, K, num_experts), experts)
    rc = lib().bsfp8_dispatch_plan(pe, pp, T, K, num_experts, *ptrs, _ptr(workspace), _stream(stream))
    _check(rc, "dispatch_plan")
    return out


def _plan_rows(plan):
    """A plan's rows and what they say: their pointer, the tokens, top_k and the rows that a buffer for them has."""
    p, (T, K) = _matrix(plan["rows"], "plan['rows']", _I32)
    return p, T, K, T * K


def dispatch(x, plan, weights=None, out=None, stream=None):
    """bsfp8_dispatch: the rows of x [tokens, cols] (fp32 or bf16) at their experts' places, out [tokens * top_k, cols],
    times weights (fp32 [tokens, top_k] or None).  Rows past the plan's last are left as they are."""
    if _elsewhere(stream):
        with _on(stream):
            return dispatch(x, plan, weights, out)
    if _use_native():
        got = _native.dispatch(*_here(), x, plan["rows"], weights, out)
        if _native_done(got, "dispatch"):
            return got[0]
    pr, T, K, N = _plan_rows(plan)
    px, (_, C) = _matrix(x, "x", _STREAM)
    _like(x, (T, C), "x")
    pw = _arg(weights, "weights", _F32, (T, K))
    if out is None:
        out = x.new_empty((N, C))
    po = _arg(out, "out", (x.dtype,), (N, C))
    _check(lib().bsfp8_dispatch(px, _dtype_code(x), T, C, pr, K, pw, po, N, _stream(stream)), "dispatch")
    return out


def dispatch_quantize(x, plan, recipe, which, out, weights=None, status=None, stream=None):
    """bsfp8_dispatch_quantize: the same rows of bf16 x [tokens, cols] quantized with an MX recipe into the layouts
    ``which`` of ``out`` (alloc_quantized for [tokens * top_k, cols] and the plan's experts), without a copy of them in
    between."""
    if _elsewhere(stream):
        with _on(stream):
            return dispatch_quantize(x, plan, recipe, which, out, weights, status)
    if _use_native() and _native_done(_native.dispatch_quantize(
            *_here(), x, plan["rows"], plan["choices"], plan["splits"], recipe, which, out.get("row_q"), out.get("row_s"),
            out.get("col_q"), out.get("col_s"), weights, status), "dispatch_quantize"):
        return out
    _, T, K, N = _plan_rows(plan)
    px, (_, C) = _matrix(x, "x", _BF16)
    _like(x, (T, C), "x")
    splits, choices = plan["splits"], plan["choices"]
    E = int(splits.numel())
    args = (px, T, C, _arg(choices, "plan['choices']", _I32, (N,)), K, _arg(weights, "weights", _F32, (T, K)), N,
            _arg(splits, "plan['splits']", _I32), E, recipe, which, _layout(out, "row_q", "out"),
            _layout(out, "row_s", "out"), _layout(out, "col_q", "out"), _layout(out, "col_s", "out"),
            _arg(status, "status", _I32))
    _need_quant(out, recipe, N, C, max(E, 1), which, "out")
    _check(lib().bsfp8_dispatch_quantize(*args, _stream(stream)), "dispatch_quantize")
    return out


def combine(y, plan, weights=None, add=None, out=None, stream=None):
    """bsfp8_combine: out[t] = add[t] + sum_j weights[t, j] * y[plan["rows"][t, j]] of y [tokens * top_k, cols] (fp32 or
    bf16), in y's type; weights fp32 [tokens, top_k] or None (1), add [tokens, cols] or None (may be out)."""
    if _elsewhere(stream):
        with _on(stream):
            return combine(y, plan, weights, add, out)
    if _use_native():
        got = _native.combine(*_here(), y, plan["rows"], weights, add, out)
        if _native_done(got, "combine"):
            return got[0]
    pr, T, K, N = _plan_rows(plan)
    py, (_, C) = _matrix(y, "y", _STREAM)
    _like(y, (N, C), "y")
    pw, pa = _arg(weights, "weights", _F32, (T, K)), _arg(add, "add", (y.dtype,), (T, C))
    if out is None:
        out = y.new_empty((T, C))
    po = _arg(out, "out", (y.dtype,), (T, C))
    _check(lib().bsfp8_combine(py, _dtype_code(y), N, C, pr, T, K, pw, pa, po, _stream(stream)), "combine")
    return out


def combine_grad(dout, plan, y=None, weights=None, dy=None, dweights=None, stream=None):
    """bsfp8_combine_grad: from dout [tokens, cols], dy [tokens * top_k, cols] of its type (the given tensor or a new one;
    False: not wanted, where dispatch_quantize makes it) and, with weights and the y [tokens * top_k, cols] that they
    were applied to, dweights (fp32 [tokens, top_k]).  Returns a dict of those.  Rows of dy past the plan's last are left
    as they are."""
    if _elsewhere(stream):
        with _on(stream):
            return combine_grad(dout, plan, y, weights, dy, dweights)
    if _use_native():
        got = _native.combine_grad(*_here(), dout, plan["rows"], y, weights, None if dy is False else dy, dy is not False,
                                   dweights)
        if _native_done(got, "combine_grad"):
            out = {"dy": got[0]} if got[0] is not None else {}
            if got[1] is not None:
                out["dweights"] = got[1]
            return out
    pr, T, K, N = _plan_rows(plan)
    pd, (_, C) = _matrix(dout, "dout", _STREAM)
    _like(dout, (T, C), "dout")
    py, pw = _arg(y, "y", (dout.dtype,), (N, C)), _arg(weights, "weights", _F32, (T, K))
    out = {}
    if dy is None:
        dy = dout.new_empty((N, C))
    if dy is not False:
        out["dy"] = dy
    if weights is not None and y is not None and dweights is None:
        dweights = torch.empty_like(weights)
    if dweights is not None:
        if y is None:
            raise ValueError("combine_grad: dweights need y")
        out["dweights"] = dweights
    rc = lib().bsfp8_combine_grad(pd, _dtype_code(dout), T, C, py, N, pr, K, pw,
                                  _arg(out.get("dy"), "dy", (dout.dtype,), (N, C)),
                                  _arg(dweights, "dweights", _F32, (T, K)), _stream(stream))
    _check(rc, "combine_grad")
    return out


# ------------------------------------------------------------------------------------------
# activations kept in 8 bits
# ------------------------------------------------------------------------------------------

def grouped_act_checkpoint(activation, h, split_sizes, recipe, which, out, kept, probs=None, status=None, stream=None):
    """bsfp8_grouped_act_checkpoint: as grouped_act_quantize with ACT_SRELU (h [R, C] bf16) or ACT_SWIGLU (h [R, 2F]), and
    in the same pass h itself in 8 bits into ``kept`` (alloc_quantized for h's shape, RECIPE_MX, ROWWISE), which is what
    grouped_act_checkpoint_grad needs of it."""
    if _elsewhere(stream):
        with _on(stream):
            return grouped_act_checkpoint(activation, h, split_sizes, recipe, which, out, kept, probs, status)
    if _use_native() and _native_done(_native.act_checkpoint(
            *_here(), activation, h, probs, split_sizes, recipe, which, out.get("row_q"), out.get("row_s"), out.get("col_q"),
            out.get("col_s"), kept.get("row_q"), kept.get("row_s"), status), "grouped_act_checkpoint"):
        return out
    ph, (R, wide) = _matrix(h, "h", _BF16)
    if activation == ACT_SWIGLU and wide % 2:
        raise ValueError("grouped_act_checkpoint: a GLU input has an even number of columns")
    F = wide // 2 if activation == ACT_SWIGLU else wide
    E = int(split_sizes.numel())
    args = (activation, ph, _arg(probs, "probs", _F32, (R,)), R, F, _arg(split_sizes, "split_sizes", _I32), E, recipe,
            which, _layout(out, "row_q", "out"), _layout(out, "row_s", "out"), _layout(out, "col_q", "out"),
            _layout(out, "col_s", "out"), _layout(kept, "row_q", "kept"), _layout(kept, "row_s", "kept"),
            _arg(status, "status", _I32))
    _need_quant(out, recipe, R, F, max(E, 1), which, "out")
    _need_quant(kept, RECIPE_MX, R, wide, 1, ROWWISE, "kept")
    _check(lib().bsfp8_grouped_act_checkpoint(*args, _stream(stream)), "grouped_act_checkpoint")
    return out


def grouped_act_checkpoint_grad_workspace_bytes(capacity_rows, cols):
    return int(lib().bsfp8_grouped_act_checkpoint_grad_workspace_bytes(capacity_rows, cols))


def grouped_act_checkpoint_grad(activation, kept, dy, split_sizes, recipe, which, out, probs=None, y=None, dprobs=None,
                                workspace=None, status=None, stream=None):
    """bsfp8_grouped_act_checkpoint_grad: from ``kept`` and the bf16 gradient dy [R, F] at the activation's output, the
    gradient at its input quantized into the layouts ``which`` (0: none) of ``out`` (alloc_quantized for [R, F] with
    ACT_SRELU, [R, 2F] with ACT_SWIGLU).  y: a dict with col_q and col_s (alloc_quantized for [R, F], COLWISE) that
    receives the activation again, for the second projection's weight gradient.  dprobs: fp32 [R], receives the
    gradient of the probabilities.  Returns a dict of out's tensors, y and dprobs, where given."""
    if _elsewhere(stream):
        with _on(stream):
            return grouped_act_checkpoint_grad(activation, kept, dy, split_sizes, recipe, which, out, probs, y, dprobs,
                                               workspace, status)
    out, q = dict(out or {}), y or {}
    if _use_native() and _native_done(_native.act_checkpoint_grad(
            *_here(), activation, kept.get("row_q"), kept.get("row_s"), dy, probs, split_sizes, recipe, which,
            out.get("row_q"), out.get("row_s"), out.get("col_q"), out.get("col_s"), q.get("col_q"), q.get("col_s"), dprobs,
            workspace, status), "grouped_act_checkpoint_grad"):
        return _glu_result(out, y=y, dprobs=dprobs)
    pd, (R, F) = _matrix(dy, "dy", _BF16)
    wide = 2 * F if activation == ACT_SWIGLU else F
    E = int(split_sizes.numel())
    args = (activation, _layout(kept, "row_q", "kept"), _layout(kept, "row_s", "kept"), _arg(probs, "probs", _F32, (R,)), pd,
            R, F, _arg(split_sizes, "split_sizes", _I32), E, recipe, which, _layout(out, "row_q", "out"),
            _layout(out, "row_s", "out"), _layout(out, "col_q", "out"), _layout(out, "col_s", "out"),
            _layout(q, "col_q", "y"), _layout(q, "col_s", "y"), _arg(dprobs, "dprobs", _F32, (R,)))
    _need_quant(kept, RECIPE_MX, R, wide, 1, ROWWISE, "kept")
    _need_quant(out, recipe, R, wide, max(E, 1), which, "out")
    if y is not None:
        _need_quant(q, recipe, R, F, max(E, 1), COLWISE, "y")
    if dprobs is not None:
        workspace = _workspace(workspace, grouped_act_checkpoint_grad_workspace_bytes(R, F), dy)
    rc = lib().bsfp8_grouped_act_checkpoint_grad(*args, _ptr(workspace) if dprobs is not None else None,
                                                 _arg(status, "status", _I32), _stream(stream))
    _check(rc, "grouped_act_checkpoint_grad")
    return _glu_result(out, y=y, dprobs=dprobs)
