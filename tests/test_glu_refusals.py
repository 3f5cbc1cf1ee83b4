"""What the fused gated projection refuses, before any HIP call (no GPU needed): the fake pointers are
never dereferenced."""
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

P = 1 << 20
OK, NULL, GROUPS, RECIPE, SHAPE, ALIGN, LAYOUT, ARG = 0, -1, -2, -3, -4, -5, -6, -7
BOTH = bs.ROWWISE | bs.COLWISE

COMMON = [
    (dict(rows=-1), SHAPE), (dict(hidden=0), SHAPE), (dict(hidden=48), SHAPE), (dict(ffn=40), SHAPE),
    (dict(ffn=(1 << 20) + 32), SHAPE), (dict(hidden=1 << 24), SHAPE), (dict(E=0), GROUPS), (dict(E=1025), GROUPS),
    (dict(recipe=9), RECIPE), (dict(recipe=bs.RECIPE_PC), LAYOUT), (dict(recipe=bs.RECIPE_MX4), LAYOUT),
    (dict(recipe=bs.RECIPE_MX | bs.GEMM_FP8_MFMA), LAYOUT), (dict(which=4), ARG), (dict(x=None), NULL),
    (dict(xs=None), NULL), (dict(w=None), NULL), (dict(ws=None), NULL), (dict(splits=None), NULL),
    (dict(rq=None), NULL), (dict(rs=None), NULL), (dict(cq=None), NULL), (dict(cs=None), NULL),
    (dict(x=P + 8), ALIGN), (dict(xs=P + 4), ALIGN), (dict(w=P + 1), ALIGN), (dict(ws=P + 2), ALIGN),
    (dict(probs=P + 2), ALIGN), (dict(splits=P + 1), ALIGN), (dict(ab=P + 8), ALIGN), (dict(rq=P + 8), ALIGN),
    (dict(cs=P + 8), ALIGN), (dict(status=P + 2), ALIGN), (dict(rows=0, x=None, w=None, splits=None), OK),
]


def forward(rows=4, hidden=64, ffn=64, E=2, x=P, xs=P, w=P, ws=P, probs=P, splits=P, recipe=bs.RECIPE_MX, ab=P, y=P,
            dtype=bs.OUT_BF16, which=BOTH, rq=P, rs=P, cq=P, cs=P, status=P):
    return bs.lib().bsfp8_grouped_gemm_swiglu(x, xs, rows, hidden, w, ws, ffn, probs, splits, E, recipe, ab, y, dtype,
                                              which, rq, rs, cq, cs, status, None)


@pytest.mark.parametrize("change,code", COMMON + [(dict(dtype=2), ARG), (dict(y=P + 8), ALIGN),
                                                  (dict(ab=None, y=None, which=0), ARG)])
def test_forward_refuses(change, code):
    assert forward(**change) == code


def grad(rows=4, hidden=64, ffn=512, E=2, x=P, xs=P, w=P, ws=P, probs=P, splits=P, recipe=bs.RECIPE_MX, ab=P, dab=P,
         which=BOTH, rq=P, rs=P, cq=P, cs=P, dp=P, work=P, status=P):
    return bs.lib().bsfp8_grouped_gemm_swiglu_grad(x, xs, rows, hidden, w, ws, ffn, ab, probs, splits, E, recipe, dab,
                                                   which, rq, rs, cq, cs, dp, work, status, None)


@pytest.mark.parametrize("change,code", COMMON + [(dict(ab=None), NULL), (dict(work=None), NULL), (dict(dp=P + 2), ALIGN),
                                                  (dict(work=P + 4), ALIGN), (dict(dab=P + 8), ALIGN),
                                                  (dict(dab=None, which=0, dp=None), ARG)])
def test_gradient_refuses(change, code):
    assert grad(**change) == code


def test_workspace_bytes():
    size = bs.grouped_gemm_swiglu_grad_workspace_bytes
    assert size(-1, 64, 2) == 0 and size(4, 40, 2) == 0 and size(4, 64, 0) == 0 and size(0, 4096, 2) == 0
    assert size(100, 4096, 2) >= 100 * 4 * 2
    assert size(200, 4096, 2) == 2 * size(100, 4096, 2) or size(200, 4096, 2) > 0


def test_binding_checks():
    """Wrong element types, host memory and short buffers are refused before the library is called."""
    q = {"row_q": torch.zeros((4, 64), dtype=torch.uint8), "row_s": torch.zeros((2, 4), dtype=torch.uint8)}
    splits = torch.tensor([4], dtype=torch.int32)
    with pytest.raises(ValueError, match="device memory"):
        bs.grouped_gemm_swiglu(q, 64, q, 64, splits, 4, y=None, out=None, stream=0)
    bad = {"row_q": torch.zeros((4, 64)), "row_s": q["row_s"]}
    with pytest.raises(TypeError, match="x_q"):
        bs.grouped_gemm_swiglu(bad, 64, q, 64, splits, 4, stream=0)
    with pytest.raises(TypeError, match="dy_q"):
        bs.grouped_gemm_swiglu_grad(bad, 64, q, 64, None, splits, 4, stream=0)
