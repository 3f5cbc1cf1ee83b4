"""What the residual norms and the AdamW step refuse, before any HIP call (no GPU needed): the fake
pointers are never dereferenced."""
import ctypes

import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

P = 1 << 20
OK, NULL, SHAPE, ALIGN, ARG = 0, -1, -4, -5, -7


def norm(rows=4, cols=64, x=P, dtype=bs.BF16, y=P, post=P, pre=P, gate=P, kind=bs.GATE_CHANNEL, xs=1.0, ys=1.0,
         eps=1e-6, off=0.0, r=P, n=P, ry=P, rr=P):
    return bs.lib().bsfp8_residual_norm(rows, cols, x, dtype, y, post, pre, gate, kind, xs, ys, eps, off, r, n, ry, rr,
                                        None)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE), (dict(cols=32769), SHAPE), (dict(dtype=2), ARG),
    (dict(eps=-1.0), ARG), (dict(eps=float("nan")), ARG), (dict(xs=float("inf")), ARG), (dict(ys=float("nan")), ARG),
    (dict(off=float("inf")), ARG), (dict(kind=3), ARG), (dict(kind=-1), ARG), (dict(kind=bs.GATE_NONE), ARG),
    (dict(gate=None), NULL), (dict(x=None), NULL), (dict(n=None), NULL),
    (dict(pre=None), ARG), (dict(pre=None, n=None), ARG), (dict(pre=None, n=None, rr=None, r=None), NULL),
    (dict(post=None), ARG), (dict(y=None), ARG), (dict(x=P + 2), ALIGN), (dict(y=P + 8), ALIGN),
    (dict(post=P + 4), ALIGN), (dict(r=P + 8), ALIGN), (dict(n=P + 2), ALIGN), (dict(rr=P + 2), ALIGN),
    (dict(rows=0, x=None, y=None, gate=None), OK),
])
def test_residual_norm_refuses(change, code):
    assert norm(**change) == code


def norm_grad(rows=4, cols=64, dtype=bs.BF16, dn=P, dr=P, r=P, rr=P, pre=P, y=P, ry=P, post=P, gate=P,
              kind=bs.GATE_CHANNEL, xs=1.0, ys=1.0, off=0.0, dx=P, dy=P, dpre=P, dpost=P, dgate=P, acc=0, ws=P):
    return bs.lib().bsfp8_residual_norm_grad(rows, cols, dtype, dn, dr, r, rr, pre, y, ry, post, gate, kind, xs, ys,
                                             off, dx, dy, dpre, dpost, dgate, acc, ws, None)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE), (dict(cols=1 << 16), SHAPE), (dict(dtype=-1), ARG),
    (dict(acc=2), ARG), (dict(xs=float("nan")), ARG), (dict(kind=3), ARG), (dict(kind=0), ARG),
    (dict(gate=None), NULL), (dict(dn=None, dr=None), NULL), (dict(r=None), NULL), (dict(rr=None), NULL),
    (dict(pre=None), NULL), (dict(ry=None), NULL), (dict(ws=None), NULL), (dict(dn=None), ARG),
    (dict(dn=None, r=None, rr=None, pre=None), ARG), (dict(y=None), ARG), (dict(post=None), ARG),
    (dict(y=None, post=None, gate=None, kind=0, dgate=None, dpost=None), ARG),
    (dict(kind=0, gate=None), ARG), (dict(dn=P + 4), ALIGN), (dict(dx=P + 4), ALIGN), (dict(dgate=P + 4), ALIGN),
    (dict(ws=P + 8), ALIGN),
])
def test_residual_norm_grad_refuses(change, code):
    assert norm_grad(**change) == code


def test_residual_norm_workspace_bytes():
    size = bs.residual_norm_grad_workspace_bytes
    assert size(-1, 64) == 0 and size(4, 0) == 0 and size(0, 64) == 0
    assert 0 < size(1, 7) <= size(100000, 7)
    assert size(1 << 30, 7168) == size(1 << 20, 7168)  # bounded in the rows


def step(plan=P, n=1, chunks=1, pd=0, gd=0, st=0, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, t=1, lr_dev=None,
         step_dev=None, gs=None, noop=None):
    return bs.lib().bsfp8_adamw_step(plan, n, chunks, pd, gd, st, lr, b1, b2, eps, wd, t, lr_dev, step_dev, gs, noop,
                                     None)


@pytest.mark.parametrize("change,code", [
    (dict(pd=2), ARG), (dict(gd=-1), ARG), (dict(st=2), ARG), (dict(lr=-1.0), ARG), (dict(lr=float("nan")), ARG),
    (dict(b1=1.0), ARG), (dict(b2=-0.1), ARG), (dict(b2=float("nan")), ARG), (dict(eps=-1e-9), ARG),
    (dict(wd=float("inf")), ARG), (dict(t=0), ARG), (dict(n=0), SHAPE), (dict(chunks=-1), SHAPE),
    (dict(chunks=1 << 31), SHAPE), (dict(plan=None), NULL), (dict(plan=P + 8), ALIGN), (dict(gs=P + 2), ALIGN),
    (dict(step_dev=P + 1), ALIGN), (dict(chunks=0, plan=None), OK),
])
def test_adamw_step_refuses(change, code):
    assert step(**change) == code


def plan_code(q8=False, pd=0, gd=0, size=None, **change):
    t = (bs._AdamTensor * 1)()
    f = dict(param=P, grad=P, exp_avg=P, exp_avg_sq=P, exp_avg_scale=P if q8 else None,
             exp_avg_sq_scale=P if q8 else None, copy=P, numel=100, lr_scale=1.0, decay_scale=1.0)
    f.update(change)
    t[0] = bs._AdamTensor(*f.values())
    buf = ctypes.create_string_buffer(4096)
    return bs.lib().bsfp8_adamw_plan(t, 1, pd, gd, 1 if q8 else 0, buf, 4096 if size is None else size)


@pytest.mark.parametrize("change,code", [
    ({}, OK), (dict(q8=True), OK), (dict(param=None), NULL), (dict(grad=None), NULL), (dict(exp_avg=None), NULL),
    (dict(q8=True, exp_avg_sq_scale=None), NULL), (dict(param=P + 2), ALIGN), (dict(param=P + 2, pd=1), OK),
    (dict(grad=P + 1, gd=1), ALIGN), (dict(exp_avg=P + 1, q8=True), OK), (dict(exp_avg=P + 1), ALIGN),
    (dict(copy=P + 1), ALIGN), (dict(copy=None), OK), (dict(numel=-1), SHAPE), (dict(numel=1 << 41), SHAPE),
    (dict(numel=0, param=None, grad=None), OK), (dict(lr_scale=float("nan")), ARG), (dict(pd=3), ARG),
    (dict(size=64), SHAPE),
])
def test_adamw_plan_refuses(change, code):
    assert plan_code(**change) == code


def test_adamw_plan_lists_every_chunk_once():
    sizes = [1, 0, 2048, 2049, 5000]
    n = len(sizes)
    numels, chunks = (ctypes.c_int64 * n)(*sizes), ctypes.c_int64()
    nbytes = bs.lib().bsfp8_adamw_plan_bytes(numels, n, ctypes.byref(chunks))
    t = (bs._AdamTensor * n)(*[bs._AdamTensor(P, P, P, P, None, None, None, s, 1.0, 1.0) for s in sizes])
    buf = ctypes.create_string_buffer(nbytes)
    assert bs.lib().bsfp8_adamw_plan(t, n, 0, 0, 0, buf, nbytes) == OK
    at = nbytes - 8 * chunks.value
    got = [tuple((ctypes.c_int32 * 2).from_buffer(buf, at + 8 * i)) for i in range(chunks.value)]
    per = 2048  # elements of a chunk
    assert got == [(i, j) for i, s in enumerate(sizes) for j in range((s + per - 1) // per)]
    assert bs.lib().bsfp8_adamw_plan_bytes((ctypes.c_int64 * 1)(-1), 1, ctypes.byref(chunks)) == 0
    assert chunks.value == 0


def test_binding_refuses_host_tensors_types_and_shapes():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64)
    with pytest.raises(ValueError, match="device memory"):
        bs.residual_norm(x, pre_weight=w)
    with pytest.raises(TypeError, match="x: dtype"):
        bs.residual_norm(x.half(), pre_weight=w)
    with pytest.raises(ValueError, match="rows, cols"):
        bs.residual_norm(x[0])
    with pytest.raises(ValueError, match="neither"):
        bs.residual_norm_grad(None, None)
    with pytest.raises(TypeError, match="dn: dtype"):
        bs.residual_norm_grad(x.float(), x)
    one = [torch.zeros(8)]
    with pytest.raises(ValueError, match="no tensors"):
        bs.adamw_plan([], [], [], [])
    with pytest.raises(ValueError, match="come together"):
        bs.adamw_plan(one, one, one, one, exp_avg_scales=one)
    with pytest.raises(ValueError, match="2 grads for 1 params"):
        bs.adamw_plan(one, one * 2, one, one)
    with pytest.raises(TypeError, match="params"):
        bs.adamw_plan([torch.zeros(8, dtype=torch.float16)], one, one, one)
    with pytest.raises(ValueError, match="device memory"):
        bs.adamw_plan(one, one, one, one)
