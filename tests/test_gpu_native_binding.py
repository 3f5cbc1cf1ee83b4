"""The native host path of the residual norms and the gated projection: the same outputs, tensors and errors as
the ctypes path, which it hands everything to that it does not take."""
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def norm_args(rows=5, cols=136, stream=torch.bfloat16, gate=bs.GATE_CHANNEL):
    g = torch.Generator(device=DEV).manual_seed(rows + cols)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    s = dict(x=rand(rows, cols).to(stream), y=rand(rows, cols).bfloat16(), post_weight=rand(cols), pre_weight=rand(cols))
    if gate != bs.GATE_NONE:
        s.update(gate=rand(cols if gate == bs.GATE_CHANNEL else rows), gate_kind=gate)
    return s


def both(monkeypatch, call):
    native = call()
    with monkeypatch.context() as m:
        m.setattr(bs, "_native", None)
        return native, call()


def same(a, b):
    assert list(a) and set(a) == set(b)
    for k in a:
        assert a[k].dtype == b[k].dtype and a[k].shape == b[k].shape and torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", [bs.GATE_NONE, bs.GATE_CHANNEL, bs.GATE_TOKEN])
@pytest.mark.parametrize("without", [(), ("post_weight",), ("pre_weight",), ("y", "post_weight", "gate", "gate_kind")])
def test_norms(monkeypatch, stream, gate, without):
    s = {k: v for k, v in norm_args(stream=stream, gate=gate).items() if k not in without}
    kw = dict(x_scale=0.5, y_scale=2.0, weight_offset=1.0)
    a, b = both(monkeypatch, lambda: bs.residual_norm(**s, eps=1e-5, **kw))
    same(a, b)
    x = s.pop("x")
    dn = x.bfloat16() if "pre_weight" in s else None
    grad = dict(s, dr=x, **kw)
    if dn is not None:
        grad.update(dn=dn, r=a["r"], rstd_r=a["rstd_r"])
    else:
        grad.update(dn=None)
    if "rstd_y" in a:
        grad.update(rstd_y=a["rstd_y"])
    same(*both(monkeypatch, lambda: bs.residual_norm_grad(**grad)))


def test_norms_given_outputs_and_accumulate():
    s = norm_args()
    out = {k: torch.empty_like(v) for k, v in bs.residual_norm(**s).items()}
    got = bs.residual_norm(**s, **out)
    assert all(got[k] is out[k] for k in out)
    grad = dict(dn=s["y"], dr=s["x"], r=got["r"], rstd_r=got["rstd_r"], rstd_y=got["rstd_y"],
                **{k: s[k] for k in ("pre_weight", "y", "post_weight", "gate", "gate_kind")})
    one = bs.residual_norm_grad(**grad)
    sums = {k: torch.ones_like(one[k]) for k in ("dpre_weight", "dpost_weight", "dgate")}
    two = bs.residual_norm_grad(**grad, **sums, accumulate=True)
    for k in sums:
        assert two[k] is sums[k] and torch.equal(two[k], one[k] + 1), k
    with pytest.raises(ValueError, match="accumulate"):
        bs.residual_norm_grad(**grad, accumulate=True)


def test_norm_errors():
    s = norm_args()
    for change, error, match in ((dict(y=s["y"].float()), TypeError, "y: dtype"), (dict(y=s["y"][:, :8]), ValueError, "y"),
                                 (dict(gate=s["gate"][:8]), ValueError, "gate"), (dict(x=s["x"].t()), ValueError, "x"),
                                 (dict(post_weight=s["post_weight"].cpu()), ValueError, "device memory"),
                                 (dict(eps=-1.0), bs.BSFP8Error, "invalid"), (dict(gate_kind=7), bs.BSFP8Error, "invalid"),
                                 (dict(n=s["y"][:2]), ValueError, "n:"), (dict(x=s["x"][0]), ValueError, "rows, cols")):
        with pytest.raises(error, match=match):
            bs.residual_norm(**dict(s, **change))


def glu_args(tokens=9, hidden=96, ffn=64, experts=3):
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn((tokens, hidden), generator=g, device=DEV).bfloat16()
    w = torch.randn((experts * 2 * ffn, hidden), generator=g, device=DEV).bfloat16()
    w2 = torch.randn((experts * hidden, ffn), generator=g, device=DEV).bfloat16()
    splits = torch.tensor([4, 0, 5], dtype=torch.int32, device=DEV)
    q = lambda t, s, which, e: bs.grouped_quantize(  # noqa: E731
        t, s, bs.RECIPE_MX, which, bs.alloc_quantized(*t.shape, e, bs.RECIPE_MX, which))
    return dict(x_q=q(x, splits, bs.ROWWISE, experts), hidden=hidden, w_q=q(w, None, bs.ROWWISE, 1), ffn=ffn,
                split_sizes=splits, capacity_rows=tokens), q(w2, torch.full((experts,), hidden, dtype=torch.int32, device=DEV),
                                                            bs.COLWISE, experts)


def test_gated_projection(monkeypatch):
    s, w2 = glu_args()
    T, F, both_ways = 9, 64, bs.ROWWISE | bs.COLWISE
    probs = torch.rand(T, device=DEV)

    def forward():
        out = bs.alloc_quantized(T, F, 3, bs.RECIPE_MX, both_ways)
        for t in out.values():
            t.zero_()
        return bs.grouped_gemm_swiglu(**s, probs=probs, ab=torch.zeros((T, 2 * F), dtype=torch.bfloat16, device=DEV),
                                      y=torch.zeros((T, F), device=DEV), y_dtype=bs.OUT_F32, out=out)

    a, b = both(monkeypatch, forward)
    same(a, b)

    def backward():
        out = bs.alloc_quantized(T, 2 * F, 3, bs.RECIPE_MX, both_ways)
        for t in out.values():
            t.zero_()
        return bs.grouped_gemm_swiglu_grad(s["x_q"], 96, w2, F, a["ab"], s["split_sizes"], T, probs=probs, out=out,
                                           dab=torch.zeros((T, 2 * F), dtype=torch.bfloat16, device=DEV),
                                           dprobs=torch.zeros(T, device=DEV))

    same(*both(monkeypatch, backward))


def test_gated_projection_errors():
    s, w2 = glu_args()
    y = torch.empty((9, 64), dtype=torch.bfloat16, device=DEV)
    short = {k: v[:1] for k, v in s["x_q"].items()}
    for change, error, match in ((dict(x_q=short), ValueError, "x_q"), (dict(y=y[:3]), ValueError, "y: "),
                                 (dict(split_sizes=s["split_sizes"].long()), TypeError, "split_sizes"),
                                 (dict(probs=torch.rand(9)), ValueError, "device memory"), (dict(y=y.float()), TypeError, "y: "),
                                 (dict(hidden=48), bs.BSFP8Error, "multiple of 32"), (dict(recipe=9), bs.BSFP8Error, "recipe"),
                                 (dict(y=None), bs.BSFP8Error, "invalid")):
        with pytest.raises(error, match=match):
            bs.grouped_gemm_swiglu(**dict(dict(s, y=y), **change))
    with pytest.raises(ValueError, match="workspace"):
        bs.grouped_gemm_swiglu_grad(s["x_q"], 96, w2, 64, torch.zeros((9, 128), dtype=torch.bfloat16, device=DEV),
                                    s["split_sizes"], 9, dprobs=torch.zeros(9, device=DEV),
                                    workspace=torch.zeros(1, dtype=torch.uint8))


def test_native_path_is_the_one_that_runs():
    s = norm_args()
    assert bs._native is not None
    assert bs._native.residual_norm(s["x"], s["y"], s["post_weight"], s["pre_weight"], s["gate"], s["gate_kind"], 1.0, 1.0,
                                    1e-6, 0.0, None, None, None, None, torch.cuda.current_stream().cuda_stream) is not None
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a = bs.residual_norm(**s)
    side.synchronize()
    same(a, bs.residual_norm(**s))


@pytest.mark.parametrize("raw", [False, True])
def test_given_stream(raw):
    """With a stream given, new outputs and workspaces belong to it: busy memory of the current stream, freed while
    its work still runs, is not written over."""
    s = norm_args(rows=300, cols=520)
    f = bs.residual_norm(**s)
    grad = dict(dn=s["y"], dr=s["x"], r=f["r"], rstd_r=f["rstd_r"], rstd_y=f["rstd_y"],
                **{k: s[k] for k in ("pre_weight", "y", "post_weight", "gate", "gate_kind")})
    want = bs.residual_norm_grad(**grad)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        junk = [torch.zeros(300, 520, dtype=torch.bfloat16, device=DEV) for _ in range(8)]
        torch.cuda._sleep(2000000)
        kept = [j + 1 for j in junk]
        del junk
        at = side.cuda_stream if raw else side
        a, b = bs.residual_norm(**s, stream=at), bs.residual_norm_grad(**grad, stream=at)
        torch.cuda.synchronize()
        same(a, f)
        same(b, want)
        assert all(bool((k == 1).all()) for k in kept)
