"""Values at which the gated projection's own arithmetic can be told from its products': products that are exact, results that
are not numbers or infinite, scales at their ends.

Tolerance.  2^x and the reciprocal of the sigmoid are within 1 ulp (2 units of 2^-24), the sum between them half of one (1),
and x = a * -log2(e), its constant and its product each rounded, is off by 1.22 units of itself, which 2^x turns into 1.22 |a|
units: the sigmoid of a number next to a.  With three more products and their second order a result is within
(1.25 |a| + 12) 2^-24 of its value."""
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = torch.float8_e4m3fn
U = 2.0 ** -24
ONE = 0x38  # e4m3 1.0
# rows and outputs that take the few-rows kernel, 128 x 128 tiles with long K steps and 256 x 256 tiles
SIZES = [(120, 32), (2000, 608), (33000, 2048)]
GRADIENT_SIZES = SIZES[:2] + [(33000, 4128)]


def ones(*shape):
    return torch.full(shape, 127, dtype=torch.uint8, device=DEV)


def sg64(a):
    return 1 / (1 + torch.exp(-a))


def codes(n, g, low, high):
    """Random positive e4m3 codes of values between low and high."""
    all_ = torch.arange(1, 127, dtype=torch.uint8, device=DEV)
    v = all_.view(E4M3).float()
    some = all_[(v >= low) & (v <= high)]
    return some[torch.randint(0, len(some), (n,), generator=g, device=DEV)]


@pytest.mark.parametrize("rows,ffn", SIZES)
def test_activation_of_exact_products(rows, ffn):
    """a = +-(c1 + c2 / 64) with c1 and c2 a row's two codes, b = c3: no product or sum is rounded."""
    g = torch.Generator(device=DEV).manual_seed(rows)
    x = torch.zeros((rows, 32), dtype=torch.uint8, device=DEV)
    x[:, 0], x[:, 1], x[:, 2] = codes(rows, g, 2.0 ** -6, 80), codes(rows, g, 2.0 ** -6, 80), codes(rows, g, 0.5, 2)
    w = torch.zeros((2 * ffn, 32), dtype=torch.uint8, device=DEV)
    w[:ffn, 0], w[:ffn, 1] = ONE, torch.tensor(2.0 ** -6).to(E4M3).view(torch.uint8).to(DEV)
    w[1:ffn:2, :2] |= 0x80
    w[ffn:, 2] = ONE
    p = torch.rand(rows, generator=g, device=DEV) + 0.25
    y = torch.empty((rows, ffn), device=DEV)
    bs.grouped_gemm_swiglu({"row_q": x, "row_s": ones(1, rows)}, 32, {"row_q": w, "row_s": ones(1, 2 * ffn)}, ffn,
                           torch.tensor([rows], dtype=torch.int32, device=DEV), rows, probs=p, y=y, y_dtype=bs.OUT_F32)
    v = x.view(E4M3).double()
    a = v[:, 0] + v[:, 1] / 64
    assert torch.equal(a.float().double(), a)
    for sign, got in ((1, y[:, 0::2]), (-1, y[:, 1::2])):
        want = (p.double() * sign * a * sg64(sign * a) * v[:, 2])[:, None]
        off = (got.double() - want).abs() / want.abs()
        tol = ((1.25 * a + 12) * U)[:, None]
        assert bool((off <= tol).all()), float((off / tol).max())


@pytest.mark.parametrize("rows,ffn", GRADIENT_SIZES)
def test_gradient_of_exact_products(rows, ffn):
    """One live channel: dh = dy there and 0 elsewhere, so dprobs is one product."""
    g = torch.Generator(device=DEV).manual_seed(rows + 1)
    dy = torch.zeros((rows, 32), dtype=torch.uint8, device=DEV)
    dy[:, 3] = codes(rows, g, 2.0 ** -6, 448)
    live = ffn // 2 + 5
    w = torch.zeros((ffn, 128), dtype=torch.uint8, device=DEV)
    w[live, 3] = ONE
    ab = torch.randn((rows, 2 * ffn), generator=g, device=DEV).bfloat16()
    ab[:, live] = (torch.rand(rows, generator=g, device=DEV) * 140 - 60).bfloat16()
    p = torch.rand(rows, generator=g, device=DEV) + 0.5
    dp, dab = torch.empty(rows, device=DEV), torch.empty_like(ab)
    bs.grouped_gemm_swiglu_grad({"row_q": dy, "row_s": ones(1, rows)}, 32, {"col_q": w.view(-1), "col_s": ones(4 * ffn)}, ffn,
                                ab, torch.tensor([rows], dtype=torch.int32, device=DEV), rows, probs=p, dab=dab, dprobs=dp)
    a, b, d = ab[:, live].double(), ab[:, ffn + live].double(), dy[:, 3].view(E4M3).double()
    sg = sg64(a)
    unit = (1.25 * a.abs() + 12) * U
    want = d * a * sg * b
    assert bool(((dp.double() - want).abs() <= unit * want.abs()).all())
    want = d * p.double() * a * sg
    assert bool(((dab[:, ffn + live].double() - want).abs() <= (2.0 ** -8 + 2 * unit) * want.abs()).all())
    want, size = d * p.double() * b * sg * (1 + a * (1 - sg)), (d * p.double() * b).abs() * sg * (1 + a.abs() * (1 - sg))
    assert bool(((dab[:, live].double() - want).abs() <= 2.0 ** -8 * want.abs() + 4 * unit * size).all())
    dead = torch.ones(2 * ffn, dtype=torch.bool, device=DEV)
    dead[live] = dead[ffn + live] = False
    assert not bool(dab[:, dead].any())


def layer(rows, ffn, hidden=64):
    g = torch.Generator(device=DEV).manual_seed(3)
    st = torch.tensor([rows], dtype=torch.int32, device=DEV)
    q = lambda t, s: bs.grouped_quantize(t, s, bs.RECIPE_MX, bs.ROWWISE, bs.alloc_quantized(*t.shape, 1, bs.RECIPE_MX, bs.ROWWISE))  # noqa: E731
    xq = q(torch.randn((rows, hidden), generator=g, device=DEV).bfloat16(), st)
    wq = q(torch.randn((2 * ffn, hidden), generator=g, device=DEV).bfloat16(), None)

    def call(p):
        out = bs.alloc_quantized(rows, ffn, 1, bs.RECIPE_MX, bs.ROWWISE | bs.COLWISE)
        y = torch.empty((rows, ffn), device=DEV)
        bs.grouped_gemm_swiglu(xq, hidden, wq, ffn, st, rows, probs=p, y=y, y_dtype=bs.OUT_F32, out=out)
        kp = (rows + 127) // 128 * 128
        return y, out["row_q"], out["row_s"], out["col_q"][:ffn * kp].view(ffn, kp), out["col_s"][:ffn * kp // 32].view(-1, ffn)

    return call


def blocks(v):
    """Bytes and codes of fp32 v [..., n] in blocks of 32: the smallest power of two that takes the largest finite or
    infinite magnitude to 448 or less (2^120 for an infinity), NaN left out of it."""
    b = v.unflatten(-1, (-1, 32))
    big = torch.where(b.isnan(), 0.0, b.abs()).amax(-1)
    frac, e = torch.frexp(big)
    e = torch.where(frac == 0, -127, (e - 9 + (frac > 0.875)).clamp(-127, 127))
    e = torch.where(big.isinf(), 120, e)
    scaled = b.double() * torch.exp2(-e.double())[..., None]
    code = scaled.float().to(E4M3).view(torch.uint8)
    odd = ~b.isfinite()
    return (e + 127).to(torch.uint8), code.flatten(-2), odd.flatten(-2)


@pytest.mark.parametrize("rows,ffn", SIZES + [(33000, 1056)])
def test_quantized_values_that_are_not_finite_and_scales_at_their_ends(rows, ffn):
    """Both layouts of y, whose rows are scaled by probabilities from 0 and 2^-149 to infinity, and by NaN: a value that is
    not finite has a NaN code; a NaN leaves its block's scale to the others, an infinity makes it 2^120."""
    call = layer(rows, ffn)
    g = torch.Generator(device=DEV).manual_seed(9)
    p = torch.rand(rows, generator=g, device=DEV)
    odd = [float("nan"), float("inf"), -float("inf"), 3e38, 1e36, 1e-36, 1e-40, 1e-45, 0.0, -0.0]
    for i, v in enumerate(odd):
        p[3 + 40 * (i % 3) + i] = v
    p[rows - 1] = float("nan")
    y, row_q, row_s, col_q, col_s = call(p)
    assert bool(y.isnan().any()) and bool(y.isinf().any()) and bool((y == 0).any())

    def check(q, s, v):
        byte, code, strange = blocks(v)
        assert torch.equal(s, byte)
        assert torch.equal(q[~strange], code[~strange])
        assert bool(((q[strange] & 0x7f) == 0x7f).all())

    check(row_q, row_s.t(), y)
    tall = torch.zeros((ffn, col_q.shape[1]), device=DEV)
    tall[:, :rows] = y.t()
    check(col_q, col_s.t(), tall)
