"""The gradient of an activation kept in 8 bits is that of the values kept, step for step: the bytes that
grouped_act_quantize writes for its gradient at those values, and for the activation again.  (A kept value has four
significant bits, so bf16 holds it.)  No tolerance: the same operations in the same order."""
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

pytestmark = pytest.mark.gpu
DEV = "cuda"
MX, MX4 = bs.RECIPE_MX, bs.RECIPE_MX4
ROW, COL, BOTH = bs.ROWWISE, bs.COLWISE, bs.ROWWISE | bs.COLWISE
GRAD = {bs.ACT_SRELU: bs.ACT_SRELU_GRAD, bs.ACT_SWIGLU: bs.ACT_SWIGLU_GRAD}


def zeroed(rows, cols, experts, recipe, which):
    q = bs.alloc_quantized(rows, cols, experts, recipe, which, DEV)
    for t in q.values():
        t.zero_()
    return q


def kept_of(h, live):
    """h[:live] in 8 bits, and the values that those stand for."""
    st = torch.tensor([live], dtype=torch.int32, device=DEV)
    kept = bs.grouped_quantize(h, st, MX, ROW, zeroed(h.shape[0], h.shape[1], 1, MX, ROW))
    scale = torch.exp2(kept["row_s"].t().float() - 127).repeat_interleave(32, 1)
    return kept, (kept["row_q"].view(torch.float8_e4m3fn).float() * scale).bfloat16()


def draw(splits, cols, act, pad, seed, wide=3.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    live = sum(splits)
    rows, both = live + pad, cols * (2 if act == bs.ACT_SWIGLU else 1)
    h = (torch.randn((rows, both), generator=g, device=DEV) * wide).bfloat16()
    dy = (torch.randn((rows, cols), generator=g, device=DEV) * 0.01).bfloat16()
    p = torch.rand(rows, generator=g, device=DEV)
    return h, dy, p, torch.tensor(splits, dtype=torch.int32, device=DEV)


def both_ways(act, h, dy, p, st, recipe):
    """(the gradient's layouts, the activation's again) from what is kept, and from the separate calls."""
    (rows, wide), cols, experts = h.shape, dy.shape[1], st.numel()
    kept, values = kept_of(h, int(st.sum()))
    q, y = zeroed(rows, wide, experts, recipe, BOTH), zeroed(rows, cols, experts, recipe, COL)
    bs.grouped_act_checkpoint_grad(act, kept, dy, st, recipe, BOTH, q, p, y)
    want_q = bs.grouped_act_quantize(GRAD[act], values, st, recipe, BOTH, zeroed(rows, wide, experts, recipe, BOTH), p, dy)
    want_y = bs.grouped_act_quantize(act, values, st, recipe, COL, zeroed(rows, cols, experts, recipe, COL), p)
    return (q, want_q), (y, want_y)


@pytest.mark.parametrize("splits,cols,pad", [([1], 32, 0), ([200, 0, 33, 128, 1], 160, 7), ([3000, 1097], 1056, 3),
                                             ([0, 4096, 129], 2048, 0)])
@pytest.mark.parametrize("act", [bs.ACT_SRELU, bs.ACT_SWIGLU])
@pytest.mark.parametrize("recipe", [MX, MX4])
@pytest.mark.parametrize("wide", [1.0, 30.0])
def test_gradient_is_that_of_the_separate_call(splits, cols, pad, act, recipe, wide):
    """Sigmoids near 1/2 and out to their ends; a code next to the border of two shows any other arithmetic."""
    h, dy, p, st = draw(splits, cols, act, pad, 1, wide)
    for got, want in both_ways(act, h, dy, p, st, recipe):
        for name in want:
            assert torch.equal(got[name], want[name]), f"{name}: {int((got[name] != want[name]).sum())} bytes"


@pytest.mark.parametrize("act", [bs.ACT_SRELU, bs.ACT_SWIGLU])
@pytest.mark.parametrize("where", ["dy", "probs", "kept"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite_reach_an_mxfp4_blocks_scale(act, where, value):
    """4-bit codes have no NaN: it shows in the block's scale, as in the separate call.  (A kept infinity is a NaN.)"""
    h, dy, p, st = draw([300, 129], 96, act, 0, 2)
    for r, c in ((0, 0), (45, 31), (299, 64), (300, 95), (428, 33)):
        if where == "kept":
            h[r, c] = value
        elif where == "dy":
            dy[r, c] = value
        else:
            p[r] = value
    (q, want_q), (y, want_y) = both_ways(act, h, dy, p, st, MX4)
    for got, want in ((q, want_q), (y, want_y)):
        for name in want:
            assert torch.equal(got[name], want[name]), f"{name}: {int((got[name] != want[name]).sum())} bytes"
    if where != "kept" or act == bs.ACT_SWIGLU:  # (the squared ReLU of a NaN is 0)
        marked = want_q["row_s"].max()
        assert int(marked) >= 252 and int((want_q["row_s"] == marked).sum()) >= 5  # 2^125 and more


@pytest.mark.parametrize("act", [bs.ACT_SRELU, bs.ACT_SWIGLU])
def test_a_nan_keeps_its_mxfp8_code_and_its_blocks_scale(act):
    h, dy, p, st = draw([64], 64, act, 0, 3)
    at = dy.abs().view(64, 2, 32).argmin(2)[:, 0]  # no block's largest
    r = torch.arange(64, device=DEV)
    h[r, at] = h[r, at].abs() + 1  # (the squared ReLU passes it on)
    clean = both_ways(act, h, dy, p, st, MX)[0][0]
    dy[r, at] = float("nan")
    got = both_ways(act, h, dy, p, st, MX)[0][0]
    code = got["row_q"].view(torch.float8_e4m3fn).float()
    assert code[r, at].isnan().all() and int(code.isnan().sum()) == 64 * (1 if act == bs.ACT_SRELU else 2)
    same = ~code.isnan()
    assert torch.equal(got["row_q"][same], clean["row_q"][same]) and torch.equal(got["row_s"], clean["row_s"])


@pytest.mark.parametrize("act", [bs.ACT_SRELU, bs.ACT_SWIGLU])
@pytest.mark.parametrize("recipe", [MX, MX4])
@pytest.mark.parametrize("which", [BOTH, COL])
def test_several_column_tiles_a_workgroup(act, recipe, which):
    """More row tiles than launches have segments for: a workgroup's waves meet in LDS again and again.  Random values in all
    rows, uneven groups, a width that ends inside a tile; whole buffers against the separate calls, several times over."""
    splits, cols, pad = [9000, 0, 1, 12345, 127, 128, 129, 7000, 4001], 4128, 33
    h, dy, p, st = draw(splits, cols, act, pad, 4)
    (rows, wide), experts, live = h.shape, len(splits), sum(splits)
    kept = zeroed(rows, wide, experts, MX, ROW)
    q = zeroed(rows, cols, experts, recipe, which)
    want_q = bs.grouped_act_quantize(act, h, st, recipe, which, zeroed(rows, cols, experts, recipe, which), p)
    want_kept, values = kept_of(h, live)
    for _ in range(3):
        bs.grouped_act_checkpoint(act, h, st, recipe, which, q, kept, p)
        for got, want in ((q, want_q), (kept, want_kept)):
            for name in want:
                assert torch.equal(got[name], want[name]), name
                got[name].zero_()
    want_g = bs.grouped_act_quantize(GRAD[act], values, st, recipe, which, zeroed(rows, wide, experts, recipe, which), p, dy)
    want_y = bs.grouped_act_quantize(act, values, st, recipe, COL, zeroed(rows, cols, experts, recipe, COL), p)
    g, y = zeroed(rows, wide, experts, recipe, which), zeroed(rows, cols, experts, recipe, COL)
    for _ in range(3):
        bs.grouped_act_checkpoint_grad(act, want_kept, dy, st, recipe, which, g, p, y)
        for got, want in ((g, want_g), (y, want_y)):
            for name in want:
                assert torch.equal(got[name], want[name]), name
                got[name].zero_()
