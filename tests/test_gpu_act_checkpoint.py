"""Activations kept in 8 bits: the forward's bytes are those of grouped_act_quantize and of grouped_quantize; the gradient
from what was kept against the formulas in 64 bits on the values that the bytes stand for.

Tolerances.  An MXFP8 value is off by half a step, 2^-4 of it or 2^-10 of its block's scale (2^-9 is the smallest code), an
MXFP4 one by 2^-2 of it (between 1 and 1.5 a step is half of 1: half of it a quarter) or 2^-2 of the scale; what is
rounded is a product of at most six fp32 factors, the hardware's exponential and reciprocal among them (the argument
off by an ulp of up to 46): 2^-17 of its terms' sizes.  dprobs is a chain of 8 terms a lane, 3 lane steps and cols / 64
parts."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

pytestmark = pytest.mark.gpu
DEV = "cuda"
MX, MX4 = bs.RECIPE_MX, bs.RECIPE_MX4
SRELU, SWIGLU = bs.ACT_SRELU, bs.ACT_SWIGLU
E2M1 = [0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6]

SPLITS = [[1], [128], [0, 0, 5, 0], [200, 0, 33, 128, 1], [64, 65, 63, 127, 129], [1000, 300], [0]]


def codes(q, recipe):
    if recipe == MX:
        return q.view(torch.float8_e4m3fn).double()
    table = torch.tensor(E2M1, dtype=torch.float64, device=q.device)
    return torch.stack([table[(q & 15).long()], table[(q >> 4).long()]], -1).flatten(-2)


def row_values(q, recipe, live):
    s = torch.exp2(q["row_s"][:, :live].t().double() - 127).repeat_interleave(32, 1)
    return codes(q["row_q"][:live], recipe) * s, s


def col_values(q, recipe, splits, cols):
    """The live rows of a colwise layout, and each value's scale."""
    per = 2 if recipe == MX4 else 1
    v, sc, p = [], [], 0
    for k in splits:
        kp = (k + 127) // 128 * 128
        c = codes(q["col_q"][cols * p // per:cols * (p + kp) // per], recipe).view(cols, kp)
        s = torch.exp2(q["col_s"][cols * p // 32:cols * (p + kp) // 32].view(kp // 32, cols).double() - 127)
        s = s.repeat_interleave(32, 0)
        assert (c[:, k:] == 0).all()
        v.append((c.t() * s)[:k])
        sc.append(s[:k])
        p += kp
    return torch.cat(v), torch.cat(sc)


def near(got, scale, ref, size, recipe):
    rel, low = (2.0 ** -4, 2.0 ** -10) if recipe == MX else (2.0 ** -2, 2.0 ** -2)
    err = (got - ref).abs()
    tol = rel * ref.abs() + low * scale + (1 + rel) * 2.0 ** -17 * size
    assert (err <= tol).all(), f"{float((err / tol).max())} times the bound"


def draw(splits, cols, act, pad, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    live = sum(splits)
    R, wide = live + pad, cols * (2 if act == SWIGLU else 1)
    h = torch.full((R, wide), float("nan"), dtype=torch.bfloat16, device=DEV)
    dy = torch.full((R, cols), float("nan"), dtype=torch.bfloat16, device=DEV)
    p = torch.full((R,), float("nan"), device=DEV)
    h[:live] = (torch.randn((live, wide), generator=g, device=DEV) * 2).bfloat16()
    dy[:live] = torch.randn((live, cols), generator=g, device=DEV).bfloat16()
    p[:live] = torch.rand(live, generator=g, device=DEV)
    if live > 3:
        h[2] = 0
        dy[3] = 0
        h[1, :40] *= 1000
        h[0, ::7] = 40.0
        h[0, 1::7] = -40.0
    return h, dy, p, torch.tensor(splits, dtype=torch.int32, device=DEV)


def poisoned(R, cols, E, recipe, which):
    q = bs.alloc_quantized(R, cols, E, recipe, which, DEV)
    for t in q.values():
        t.fill_(0xEE)
    return q


@pytest.mark.parametrize("splits", SPLITS)
@pytest.mark.parametrize("cols,pad", [(32, 0), (128, 1), (160, 300)])
@pytest.mark.parametrize("act", [SRELU, SWIGLU])
@pytest.mark.parametrize("recipe,which,probs", [(MX, 3, True), (MX, bs.ROWWISE, False), (MX4, 3, True),
                                                (MX4, bs.COLWISE, False)])
def test_forward_bytes(splits, cols, pad, act, recipe, which, probs):
    h, _, p, st = draw(splits, cols, act, pad)
    (R, wide), E = h.shape, len(splits)
    if R == 0:
        pytest.skip("no rows")
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    p = p if probs else None
    kept = poisoned(R, wide, E, MX, bs.ROWWISE)
    got = bs.grouped_act_checkpoint(act, h, st, recipe, which, poisoned(R, cols, E, recipe, which), kept, p, status)
    want = bs.grouped_act_quantize(act, h, st, recipe, which, poisoned(R, cols, E, recipe, which), p, status=status)
    for name in want:
        assert torch.equal(got[name], want[name]), name
    want = bs.grouped_quantize(h, st, MX, bs.ROWWISE, poisoned(R, wide, E, MX, bs.ROWWISE), status=status)
    for name in want:
        assert torch.equal(kept[name], want[name]), name
    assert int(status) == 0


def formulas(kept, dy, p, act, cols, live):
    """(gradient, its terms' size, value, dprobs, its terms' size) in 64 bits from the values kept."""
    h, _ = row_values(kept, MX, live)
    dy, p = dy[:live].double(), p[:live].double()[:, None]
    if act == SRELU:
        r = h.clamp(min=0)
        g, v = 2 * r * p * dy, r * r
        size = g.abs()
    else:
        a, b = h[:, :cols], h[:, cols:]
        sg = torch.sigmoid(a)
        v = a * sg * b
        g = torch.cat([dy * p * b * sg * (1 + a * (1 - sg)), dy * p * a * sg], 1)
        size = torch.cat([(dy * p * b * sg).abs() * (1 + a.abs()), (dy * p * a * sg).abs()], 1)
    return g, size, v, (dy * v).sum(1), (dy * v).abs().sum(1)


@pytest.mark.parametrize("splits", SPLITS)
@pytest.mark.parametrize("cols,pad", [(32, 0), (64, 1), (160, 300), (1056, 5)])
@pytest.mark.parametrize("act", [SRELU, SWIGLU])
@pytest.mark.parametrize("recipe", [MX, MX4])
def test_gradient(splits, cols, pad, act, recipe):
    h, dy, p, st = draw(splits, cols, act, pad, 1)
    (R, wide), E, live = h.shape, len(splits), sum(splits)
    if R == 0:
        pytest.skip("no rows")
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    kept = poisoned(R, wide, E, MX, bs.ROWWISE)
    bs.grouped_act_checkpoint(act, h, st, recipe, bs.ROWWISE, poisoned(R, cols, E, recipe, bs.ROWWISE), kept, p, status)
    y, dp = poisoned(R, cols, E, recipe, bs.COLWISE), torch.full((R,), 99.0, device=DEV)
    q = poisoned(R, wide, E, recipe, 3)
    out = bs.grouped_act_checkpoint_grad(act, kept, dy, st, recipe, 3, q, p, y, dp, status=status)
    assert int(status) == 0 and out["dprobs"] is dp and out["y"] is y
    # nothing is written past the live rows and the groups' extents
    used = sum((k + 127) // 128 * 128 for k in splits)
    per = 2 if recipe == MX4 else 1
    assert (q["row_q"][live:] == 0xEE).all() and (q["row_s"][:, live:] == 0xEE).all() and (dp[live:] == 99).all()
    for d, w in ((q, wide), (y, cols)):
        assert (d["col_q"][used * w // per:] == 0xEE).all() and (d["col_s"][used * w // 32:] == 0xEE).all()
    if live == 0:
        return
    g, size, v, ref, terms = formulas(kept, dy, p, act, cols, live)
    near(*row_values(q, recipe, live), g, size, recipe)
    near(*col_values(q, recipe, splits, wide), g, size, recipe)
    v = v * p[:live].double()[:, None]
    near(*col_values(y, recipe, splits, cols), v, v.abs(), recipe)
    assert ((dp[:live].double() - ref).abs() <= ((11 + cols / 64) * 2.0 ** -24 + 2.0 ** -17) * terms + 1e-40).all()
    # each output alone has the same bits
    for which, names in ((bs.ROWWISE, ("row_q", "row_s")), (bs.COLWISE, ("col_q", "col_s"))):
        one = bs.grouped_act_checkpoint_grad(act, kept, dy, st, recipe, which, poisoned(R, wide, E, recipe, which), p)
        assert all(torch.equal(one[n], q[n]) for n in names)
    only = bs.grouped_act_checkpoint_grad(act, kept, dy, st, recipe, 0, None, p, poisoned(R, cols, E, recipe, bs.COLWISE))
    assert all(torch.equal(only["y"][n], y[n]) for n in y)
    dp2 = torch.full((R,), 99.0, device=DEV)
    bs.grouped_act_checkpoint_grad(act, kept, dy, st, recipe, 0, None, p, dprobs=dp2)
    assert torch.equal(dp, dp2)


@pytest.mark.parametrize("act", [SRELU, SWIGLU])
def test_gradient_is_that_of_differences(act):
    """Central differences of the activation in 64 bits at the values kept, for the inputs and the probabilities."""
    splits, cols = [40, 24], 64
    h, dy, p, st = draw(splits, cols, act, 0, 2)
    R, wide = h.shape
    kept = bs.alloc_quantized(R, wide, 2, MX, bs.ROWWISE)
    bs.grouped_act_checkpoint(act, h, st, MX, bs.ROWWISE, bs.alloc_quantized(R, cols, 2, MX, bs.ROWWISE), kept, p)
    q, dp = bs.alloc_quantized(R, wide, 2, MX, bs.ROWWISE), torch.empty(R, device=DEV)
    bs.grouped_act_checkpoint_grad(act, kept, dy, st, MX, bs.ROWWISE, q, p, dprobs=dp)
    x, _ = row_values(kept, MX, R)
    d, pp = dy.double(), p.double()[:, None]

    def value(h, prob):
        if act == SRELU:
            return (h.clamp(min=0) ** 2 * prob * d)
        return h[:, :cols] * torch.sigmoid(h[:, :cols]) * h[:, cols:] * prob * d

    step = 2.0 ** -12
    diff = []
    for half in range(wide // cols):
        e = torch.zeros_like(x)
        e[:, half * cols:(half + 1) * cols] = step
        diff.append((value(x + e, pp) - value(x - e, pp)) / (2 * step))
    diff = torch.cat(diff, 1)
    got, s = row_values(q, MX, R)
    # the third derivative (SwiGLU: below |b dy|; SReLU: the kink, 2 step |dy|) leaves 2 step^2 or 2 step of the sizes
    slack = 4 * step * d.abs().repeat(1, wide // cols) * (1 + x.abs().amax(1, keepdim=True))
    assert ((got - diff).abs() <= 2.0 ** -4 * diff.abs() + 2.0 ** -10 * s + slack).all()
    dprob = (value(x, pp + 1) - value(x, pp)).sum(1)
    size = (value(x, pp * 0 + 1)).abs().sum(1)
    assert ((dp - dprob).abs() <= 2.0 ** -16 * size + 1e-30).all()


def test_large_values_and_empty_blocks():
    """Blocks of zeros, of the largest bf16 numbers, and of the smallest: the bytes stay those of the separate calls,
    and their gradient is finite where the formula is."""
    st = torch.tensor([96], dtype=torch.int32, device=DEV)
    h = torch.zeros((96, 128), dtype=torch.bfloat16, device=DEV)
    h[0] = 3e38
    h[1] = -3e38
    h[2] = 1e-38
    h[3] = 9e-41
    h[4, ::2] = float("inf")
    h[5, 3] = float("nan")
    kept = bs.alloc_quantized(96, 128, 1, MX, bs.ROWWISE)
    got = bs.grouped_act_checkpoint(SWIGLU, h, st, MX, 3, bs.alloc_quantized(96, 64, 1, MX, 3), kept)
    want = bs.grouped_act_quantize(SWIGLU, h, st, MX, 3, bs.alloc_quantized(96, 64, 1, MX, 3))
    assert all(torch.equal(got[n], want[n]) for n in got)
    want = bs.grouped_quantize(h, st, MX, bs.ROWWISE, bs.alloc_quantized(96, 128, 1, MX, bs.ROWWISE))
    assert all(torch.equal(kept[n], want[n]) for n in kept)
    dy = torch.full((96, 64), 1e-30, dtype=torch.bfloat16, device=DEV)
    q, dp = bs.alloc_quantized(96, 128, 1, MX, bs.ROWWISE), torch.empty(96, device=DEV)
    bs.grouped_act_checkpoint_grad(SWIGLU, kept, dy, st, MX, bs.ROWWISE, q, dprobs=dp)
    g, _ = row_values(q, MX, 96)
    assert torch.isfinite(g[[1, 2, 3, 6, 95]]).all() and (g[6:] == 0).all() and (dp[6:] == 0).all()
    assert g[5].isnan().any()  # a NaN stays one


def test_bad_sizes_set_the_status_and_write_nothing():
    h, dy, p, _ = draw([64, 64], 64, SWIGLU, 0, 3)
    kept = poisoned(128, 128, 2, MX, bs.ROWWISE)
    for sizes, bit in (([-1, 4], bs.STATUS_NEGATIVE_SPLIT), ([100, 29], bs.STATUS_EXCEEDS_CAPACITY)):
        st = torch.tensor(sizes, dtype=torch.int32, device=DEV)
        status, q, dp = torch.zeros(1, dtype=torch.int32, device=DEV), poisoned(128, 64, 2, MX, 3), torch.full((128,), 9.0, device=DEV)
        bs.grouped_act_checkpoint(SWIGLU, h, st, MX, 3, q, kept, p, status)
        assert int(status) == bit and all((t == 0xEE).all() for t in (*q.values(), *kept.values()))
        status.zero_()
        q = poisoned(128, 128, 2, MX, 3)
        bs.grouped_act_checkpoint_grad(SWIGLU, kept, dy, st, MX, 3, q, p, dprobs=dp, status=status)
        assert int(status) == bit and all((t == 0xEE).all() for t in q.values()) and (dp == 9).all()
