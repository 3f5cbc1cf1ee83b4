"""The fused gated projection and its gradient against their formulas in 64 bits, from the values that
the MXFP8 operands stand for.

Tolerances.  A product of length K is off by at most one fp32 rounding for every four terms and 16
more, of the sum of its terms' sizes: t = (K / 4 + 16) 2^-24 sum |x| |w|.  silu's slope is at most
1.1, so y is off by |p| (1.1 |b| ta + |silu(a)| tb) and 16 roundings of its own; the gradients
likewise, with a + 1 for the factors in sg (1 + a (1 - sg)).  A bf16 output adds 2^-8 of its value.
Quantized values add half a step of e4m3: 2^-4 of the value, or 2^-10 of the block's scale.  Where the
fp32 result is at hand, its quantization is exact.  dprobs is a chain of at most 32 + F / 64 terms."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs
import workloads as W
from gpu_util import DEV, flush

pytestmark = pytest.mark.gpu
F64, E4M3 = torch.float64, torch.float8_e4m3fn
U = 2.0 ** -24
SPLITS = [[0, 1, 31, 32, 33, 127, 128, 129, 256], [300, 0, 45, 1, 200], [1000], [0, 0, 5], [1, 0, 1, 1], [16, 17, 40],
          [700, 3], [2]]
BOTH = bs.ROWWISE | bs.COLWISE


def deq(q, s):
    """Codes [n, k] and scales [k / 32, n] as values."""
    return q.view(E4M3).to(F64) * torch.exp2(s.t().to(F64) - 127).repeat_interleave(32, 1)


def operands(splits, hidden, ffn, seed, pad=37, scale=1.0):
    """x [R, hidden], W1 [E, 2 ffn, hidden], W2 [E, hidden, ffn] quantized as the GEMMs take them, their
    values, probs and ab, with garbage past the live rows."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    T, E = sum(splits), len(splits)
    R = T + pad
    x = W.randn_bf16((R, hidden), g, DEV, scale=scale)
    w1 = W.randn_bf16((E * 2 * ffn, hidden), g, DEV, scale=hidden ** -0.5)
    w2 = W.randn_bf16((E * hidden, ffn), g, DEV, scale=ffn ** -0.5)
    st = W.splits_tensor(splits, DEV)
    xq = bs.grouped_quantize(x, st, bs.RECIPE_MX, bs.ROWWISE, bs.alloc_quantized(R, hidden, E, bs.RECIPE_MX, bs.ROWWISE))
    w1q = bs.grouped_quantize(w1, None, bs.RECIPE_MX, bs.ROWWISE,
                              bs.alloc_quantized(E * 2 * ffn, hidden, 1, bs.RECIPE_MX, bs.ROWWISE))
    w2q = bs.grouped_quantize(w2, W.splits_tensor([hidden] * E, DEV), bs.RECIPE_MX, bs.COLWISE,
                              bs.alloc_quantized(E * hidden, ffn, E, bs.RECIPE_MX, bs.COLWISE))
    rng = np.random.default_rng(seed)
    if pad:
        xq["row_q"][T:] = torch.from_numpy(rng.integers(0, 256, (pad, hidden), dtype=np.uint8)).to(DEV)
        xq["row_s"][:, T:] = 0xFF
    ab = W.randn_bf16((R, 2 * ffn), g, DEV, scale=1.5)
    ab[T:] = float("nan")
    p = torch.rand(R, generator=g, device=DEV) - 0.25
    p[T:] = float("nan")
    hp = 128 * ((hidden + 127) // 128)
    w2v = (w2q["col_q"][:E * ffn * hp].view(E, ffn, hp).view(E4M3).to(F64)
           * torch.exp2(w2q["col_s"][:E * ffn * hp // 32].view(E, hp // 32, ffn).transpose(1, 2).to(F64) - 127)
           .repeat_interleave(32, 2))[:, :, :hidden]
    return dict(splits=splits, st=st, T=T, E=E, R=R, hidden=hidden, ffn=ffn, xq=xq, w1q=w1q, w2q=w2q, p=p, ab=ab,
                xv=deq(xq["row_q"][:T], xq["row_s"][:, :T]),
                w1v=deq(w1q["row_q"], w1q["row_s"]).view(E, 2 * ffn, hidden), w2v=w2v)


def products(s, w):
    """Each live row times its expert's w [E, n, hidden], and the sums of the terms' sizes."""
    v = torch.empty((s["T"], w.shape[1]), dtype=F64, device=DEV)
    m = torch.empty_like(v)
    at = 0
    for e, k in enumerate(s["splits"]):
        v[at:at + k] = s["xv"][at:at + k] @ w[e].t().contiguous()
        m[at:at + k] = s["xv"][at:at + k].abs() @ w[e].abs().t().contiguous()
        at += k
    return v, m * ((s["hidden"] / 4 + 16) * U)


def within(got, ref, tol, what):
    err = (got.to(F64) - ref).abs()
    bad = ~(err <= tol + 1e-30)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()}, worst {float((err / (tol + 1e-30)).max()):.3g}"


def forward64(s):
    ab, t = products(s, s["w1v"])
    f = s["ffn"]
    a, b, ta, tb = ab[:, :f], ab[:, f:], t[:, :f], t[:, f:]
    p = s["p"][:s["T"], None].to(F64) if s["p"] is not None else 1.0
    sl = a * torch.sigmoid(a)
    y = sl * b * p
    ty = abs(p) * (1.1 * b.abs() * ta + sl.abs() * tb + 1.1 * ta * tb) + 16 * U * y.abs()
    return ab, t, y, ty


def backward64(s):
    dh, t = products(s, s["w2v"])
    T, f = s["T"], s["ffn"]
    a = s["ab"][:T, :f].to(F64).requires_grad_()
    b = s["ab"][:T, f:].to(F64).requires_grad_()
    p = (torch.ones(T, dtype=F64, device=DEV) if s["p"] is None else s["p"][:T].to(F64)).requires_grad_()
    (a * torch.sigmoid(a) * b * p[:, None] * dh).sum().backward()
    a0, b0, p0 = a.detach(), b.detach(), p.detach()[:, None]
    sg = torch.sigmoid(a0)
    sl = (a0 * sg).abs()
    slope = sg * (1 + a0.abs() * (1 - sg))  # with its terms' sizes
    tda = p0.abs() * b0.abs() * slope * (t + 24 * U * dh.abs()) + p0.abs() * b0.abs() * dh.abs() * a0.abs() * sg * 8 * U
    tdb = p0.abs() * sl * (t + 16 * U * dh.abs())
    tp = (sl * b0.abs() * (t + (64 + f / 64) * U * dh.abs())).sum(1)
    return torch.cat([a.grad, b.grad], 1), torch.cat([tda, tdb], 1), p.grad, tp


def poisoned(R, cols, E, which=BOTH):
    out = bs.alloc_quantized(R, cols, E, bs.RECIPE_MX, which, DEV)
    for t in out.values():
        t.fill_(0xFF)
    return out


def packed(splits):
    kp = [(k + 127) // 128 * 128 for k in splits]
    return kp, np.cumsum([0] + kp)


def col_values(out, splits, C):
    """The colwise codes and scales of the live groups: per expert codes [C, kp] and bytes [kp / 32, C]."""
    kp, at = packed(splits)
    for e, k in enumerate(splits):
        q = out["col_q"][C * at[e]:C * at[e + 1]].view(C, kp[e])
        sc = out["col_s"][C * at[e] // 32:C * at[e + 1] // 32].view(kp[e] // 32, C)
        yield e, k, q, sc


def quantize32(v):
    """MXFP8 of fp32 [..., n] (n a multiple of 32): codes, bytes."""
    b = v.unflatten(-1, (-1, 32))
    frac, e = torch.frexp(b.abs().amax(-1))
    e = torch.where(frac == 0, -127, (e - 9 + (frac > 0.875)).clamp(-127, 127))
    q = (b * torch.exp2(-e.double()).float().unsqueeze(-1)).to(E4M3)
    return q.flatten(-2).view(torch.uint8), (e + 127).to(torch.uint8)


def check_untouched(out, s, C):
    T = s["T"]
    assert bool((out["row_q"][T:] == 0xFF).all()) and bool((out["row_s"][:, T:] == 0xFF).all())
    end = int(packed(s["splits"])[1][-1])
    assert bool((out["col_q"][C * end:] == 0xFF).all()) and bool((out["col_s"][C * end // 32:] == 0xFF).all())


def check_exact_quantization(out, y, s):
    """The codes of fp32 y, bit for bit, in both layouts."""
    T, C = s["T"], y.shape[1]
    q, sc = quantize32(y[:T])
    assert torch.equal(out["row_s"][:, :T], sc.t()) and torch.equal(out["row_q"][:T], q)
    at = 0
    for e, k, cq, cs in col_values(out, s["splits"], C):
        tall = torch.zeros((C, cq.shape[1]), device=DEV)
        tall[:, :k] = y[at:at + k].t()
        if k:
            q, sc = quantize32(tall)
            # a zero keeps the sign it was computed with in the live rows, none in the pad lanes
            assert torch.equal(cs, sc.t()) and torch.equal(cq, q), e
        at += k


def check_close_quantization(out, v, tol, s):
    """Both layouts stand for v to half a step of e4m3, their scales follow the blocks' largest."""
    T, C = s["T"], v.shape[1]

    def one(q, sc, v, tol, what):  # codes [..., n], bytes [..., n / 32]
        wide = torch.exp2(sc.to(F64) - 127)
        sw = wide.repeat_interleave(32, -1)
        within(q.view(E4M3).to(F64) * sw, v, (v.abs() + tol) * 2.0 ** -4 + sw * 2.0 ** -10 + tol, what)
        big = v.abs().unflatten(-1, (-1, 32)).amax(-1)
        more = tol.unflatten(-1, (-1, 32)).amax(-1)
        assert bool((448 * wide >= big - more - 1e-37).all()), what
        assert bool(((sc == 0) | (224 * wide <= big + more)).all()), what

    one(out["row_q"][:T], out["row_s"][:, :T].t().contiguous(), v, tol, "row")
    at = 0
    for e, k, cq, cs in col_values(out, s["splits"], C):
        if k:
            tall, tt = torch.zeros(cq.shape, dtype=F64, device=DEV), torch.zeros(cq.shape, dtype=F64, device=DEV)
            tall[:, :k], tt[:, :k] = v[at:at + k].t(), tol[at:at + k].t()
            one(cq, cs.t().contiguous(), tall, tt, f"col {e}")
            assert not bool(cq[:, k:].any()), f"pad lanes {e}"
        at += k


SIZES = [(32, 32), (160, 96), (128, 128), (416, 320), (1056, 160)]


@pytest.mark.parametrize("splits", SPLITS)
@pytest.mark.parametrize("hidden,ffn", SIZES)
def test_forward(splits, hidden, ffn):
    flush(f"{splits} {hidden} {ffn}")
    s = operands(splits, hidden, ffn, hidden + ffn + sum(splits))
    R, T = s["R"], s["T"]
    ab = torch.full((R, 2 * ffn), float("nan"), dtype=torch.bfloat16, device=DEV)
    y = torch.full((R, ffn), float("nan"), device=DEV)
    out = poisoned(R, ffn, s["E"])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    bs.grouped_gemm_swiglu(s["xq"], hidden, s["w1q"], ffn, s["st"], R, probs=s["p"], ab=ab, y=y, y_dtype=bs.OUT_F32,
                           out=out, status=status)
    assert int(status.item()) == 0
    rab, tab, ry, ty = forward64(s)
    within(ab[:T], rab, 2.0 ** -8 * rab.abs() + 1.01 * tab, "ab")
    within(y[:T], ry, ty, "y")
    assert bool(ab[T:].isnan().all()) and bool(y[T:].isnan().all())
    check_exact_quantization(out, y, s)
    check_untouched(out, s, ffn)
    # each output by itself, in bf16, the same bits
    y16 = torch.empty((R, ffn), dtype=torch.bfloat16, device=DEV)
    bs.grouped_gemm_swiglu(s["xq"], hidden, s["w1q"], ffn, s["st"], R, probs=s["p"], y=y16)
    assert torch.equal(y16[:T], y[:T].bfloat16())
    for which in (bs.ROWWISE, bs.COLWISE):
        part = poisoned(R, ffn, s["E"], which)
        bs.grouped_gemm_swiglu(s["xq"], hidden, s["w1q"], ffn, s["st"], R, probs=s["p"], out=part)
        for k, t in part.items():
            assert torch.equal(t, out[k]), k
    ab2 = torch.full_like(ab, float("nan"))
    bs.grouped_gemm_swiglu(s["xq"], hidden, s["w1q"], ffn, s["st"], R, ab=ab2)
    assert torch.equal(ab2[:T], ab[:T])


@pytest.mark.parametrize("splits", SPLITS)
@pytest.mark.parametrize("hidden,ffn", SIZES + [(96, 544)])
def test_gradient(splits, hidden, ffn):
    flush(f"{splits} {hidden} {ffn}")
    s = operands(splits, hidden, ffn, 7 + hidden + ffn + sum(splits))
    R, T = s["R"], s["T"]
    dab = torch.full((R, 2 * ffn), float("nan"), dtype=torch.bfloat16, device=DEV)
    dp = torch.full((R,), float("nan"), device=DEV)
    out = poisoned(R, 2 * ffn, s["E"])
    bs.grouped_gemm_swiglu_grad(s["xq"], hidden, s["w2q"], ffn, s["ab"], s["st"], R, probs=s["p"], dab=dab, out=out,
                                dprobs=dp)
    rd, td, rp, tp = backward64(s)
    within(dab[:T], rd, 2.0 ** -8 * rd.abs() + 1.01 * td, "dab")
    within(dp[:T], rp, tp, "dprobs")
    assert bool(dab[T:].isnan().all()) and bool(dp[T:].isnan().all())
    check_close_quantization(out, rd, td, s)
    check_untouched(out, s, 2 * ffn)
    # each output by itself, the same bits
    d2, p2 = torch.empty_like(dab), torch.empty_like(dp)
    bs.grouped_gemm_swiglu_grad(s["xq"], hidden, s["w2q"], ffn, s["ab"], s["st"], R, probs=s["p"], dab=d2)
    bs.grouped_gemm_swiglu_grad(s["xq"], hidden, s["w2q"], ffn, s["ab"], s["st"], R, probs=s["p"], dprobs=p2)
    assert torch.equal(d2[:T], dab[:T]) and torch.equal(p2[:T], dp[:T])
    for which in (bs.ROWWISE, bs.COLWISE):
        part = poisoned(R, 2 * ffn, s["E"], which)
        bs.grouped_gemm_swiglu_grad(s["xq"], hidden, s["w2q"], ffn, s["ab"], s["st"], R, probs=s["p"], out=part)
        for k, t in part.items():
            assert torch.equal(t, out[k]), k


@pytest.mark.parametrize("splits", [[3, 0, 2], [130, 70, 400]])
def test_no_probabilities(splits):
    s = operands(splits, 160, 96, 3)
    s["p"] = None
    y = torch.empty((s["R"], 96), device=DEV)
    bs.grouped_gemm_swiglu(s["xq"], 160, s["w1q"], 96, s["st"], s["R"], y=y, y_dtype=bs.OUT_F32)
    _, _, ry, ty = forward64(s)
    within(y[:s["T"]], ry, ty, "y")
    dab, dp = torch.empty((s["R"], 192), dtype=torch.bfloat16, device=DEV), torch.empty(s["R"], device=DEV)
    bs.grouped_gemm_swiglu_grad(s["xq"], 160, s["w2q"], 96, s["ab"], s["st"], s["R"], dab=dab, dprobs=dp)
    rd, td, rp, tp = backward64(s)
    within(dab[:s["T"]], rd, 2.0 ** -8 * rd.abs() + 1.01 * td, "dab")
    within(dp[:s["T"]], rp, tp, "dprobs")


@pytest.mark.parametrize("splits", [[3, 0, 2], [130, 70, 400]])
def test_saturated_activations(splits):
    """|a| far beyond the exponential's range on both sides: silu(a) is a or 0, its slope 1 or 0."""
    s = operands(splits, 160, 96, 5, scale=400.0)
    s["ab"][:s["T"], :96] *= 300
    y = torch.empty((s["R"], 96), device=DEV)
    bs.grouped_gemm_swiglu(s["xq"], 160, s["w1q"], 96, s["st"], s["R"], probs=s["p"], y=y, y_dtype=bs.OUT_F32)
    ab, _, ry, ty = forward64(s)
    assert float(ab[:, :96].abs().max()) > 300
    # below a = -87 the hardware's 2^x and its reciprocal leave fp32's normal range: 2^-126 of the terms
    within(y[:s["T"]], ry, ty + 2.0 ** -100, "y")
    dab = torch.empty((s["R"], 192), dtype=torch.bfloat16, device=DEV)
    bs.grouped_gemm_swiglu_grad(s["xq"], 160, s["w2q"], 96, s["ab"], s["st"], s["R"], probs=s["p"], dab=dab)
    rd, td, _, _ = backward64(s)
    within(dab[:s["T"]], rd, 2.0 ** -8 * rd.abs() + 1.01 * td + 2.0 ** -100, "dab")


@pytest.mark.parametrize("splits", [[2, 1, 0, 4], [200, 0, 260]])
def test_gradient_against_differences(splits):
    """dprobs and dab along random directions against central differences of the 64-bit loss; the
    differences' own error is of the third derivative, h^2 = 1e-6 of the terms."""
    s = operands(splits, 96, 64, 9)
    T = s["T"]
    dab, dp = torch.empty((s["R"], 128), dtype=torch.bfloat16, device=DEV), torch.empty(s["R"], device=DEV)
    bs.grouped_gemm_swiglu_grad(s["xq"], 96, s["w2q"], 64, s["ab"], s["st"], s["R"], probs=s["p"], dab=dab, dprobs=dp)
    dh, _ = products(s, s["w2v"])
    ab, p = s["ab"][:T].to(F64), s["p"][:T].to(F64)

    def loss(ab, p):
        return float((ab[:, :64] * torch.sigmoid(ab[:, :64]) * ab[:, 64:] * p[:, None] * dh).sum())

    g = torch.Generator(device=DEV).manual_seed(1)
    v, u, h = torch.randn(ab.shape, generator=g, device=DEV, dtype=F64), torch.randn(T, generator=g, device=DEV, dtype=F64), 1e-3
    diff = (loss(ab + h * v, p) - loss(ab - h * v, p)) / (2 * h)
    size = float((dab[:T].to(F64) * v).abs().sum())
    assert abs(diff - float((dab[:T].to(F64) * v).sum())) <= (2.0 ** -8 + 1e-4) * size
    diff = (loss(ab, p + h * u) - loss(ab, p - h * u)) / (2 * h)
    assert abs(diff - float((dp[:T].to(F64) * u).sum())) <= 1e-5 * float((dp[:T].to(F64) * u).abs().sum()) + 1e-9


def test_bad_sizes_write_nothing():
    s = operands([40, 60], 96, 64, 11)
    for splits, bit in (([-1, 20], bs.STATUS_NEGATIVE_SPLIT), ([100, 100], bs.STATUS_EXCEEDS_CAPACITY)):
        st = torch.tensor(splits, dtype=torch.int32, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        y, dp = torch.full((s["R"], 64), 7.0, device=DEV), torch.full((s["R"],), 7.0, device=DEV)
        dab = torch.full((s["R"], 128), 7.0, dtype=torch.bfloat16, device=DEV)
        bs.grouped_gemm_swiglu(s["xq"], 96, s["w1q"], 64, st, s["R"], y=y, y_dtype=bs.OUT_F32, status=status)
        assert int(status.item()) == bit and bool((y == 7).all())
        status.zero_()
        bs.grouped_gemm_swiglu_grad(s["xq"], 96, s["w2q"], 64, s["ab"], st, s["R"], dab=dab, dprobs=dp, status=status)
        assert int(status.item()) == bit and bool((dab == 7).all()) and bool((dp == 7).all())


@pytest.mark.parametrize("splits", [[4, 0, 3, 1], [300, 130, 0, 77]])
def test_graph_and_other_stream(splits):
    """Captured with all outputs, replayed with new inputs and sizes; every replay equals the eager call."""
    hidden, ffn = 160, 320
    s = operands(splits, hidden, ffn, 13)
    R, E = s["R"], s["E"]

    def outputs():
        return dict(ab=torch.zeros((R, 2 * ffn), dtype=torch.bfloat16, device=DEV), y=torch.zeros((R, ffn), device=DEV),
                    q=poisoned(R, ffn, E), dab=torch.zeros((R, 2 * ffn), dtype=torch.bfloat16, device=DEV),
                    dq=poisoned(R, 2 * ffn, E), dp=torch.zeros(R, device=DEV))

    def call(o, ws):
        bs.grouped_gemm_swiglu(s["xq"], hidden, s["w1q"], ffn, s["st"], R, probs=s["p"], ab=o["ab"], y=o["y"],
                               y_dtype=bs.OUT_F32, out=o["q"])
        bs.grouped_gemm_swiglu_grad(s["xq"], hidden, s["w2q"], ffn, o["ab"], s["st"], R, probs=s["p"], dab=o["dab"],
                                    out=o["dq"], dprobs=o["dp"], workspace=ws)

    ws = torch.zeros(max(16, bs.grouped_gemm_swiglu_grad_workspace_bytes(R, ffn, E)), dtype=torch.uint8, device=DEV)
    o = outputs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(o, ws)
    side = torch.cuda.Stream()
    for turn in range(3):
        n = operands(splits[turn:] + splits[:turn], hidden, ffn, 20 + turn)
        for k in ("st", "p"):
            s[k].copy_(n[k])
        s["xq"]["row_q"].copy_(n["xq"]["row_q"])
        s["xq"]["row_s"].copy_(n["xq"]["row_s"])
        ws.fill_(0xFF)
        for t in (o["ab"], o["y"], o["dab"], o["dp"]):
            t.zero_()
        for t in list(o["q"].values()) + list(o["dq"].values()):
            t.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        e = outputs()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call(e, torch.empty_like(ws))
        side.synchronize()
        for k in ("ab", "y", "dab", "dp"):
            assert torch.equal(o[k], e[k]), (turn, k)
        for k in ("q", "dq"):
            for name in o[k]:
                assert torch.equal(o[k][name], e[k][name]), (turn, k, name)


@pytest.mark.parametrize("splits", [[4, 0, 3, 1], [300, 130, 0, 77]])
def test_rows_do_not_depend_on_their_neighbours(splits):
    """A row's y is the same bits with other probabilities, padding and capacity (within one kernel)."""
    s = operands(splits, 416, 96, 17)
    T, R = s["T"], s["R"]
    y = torch.empty((R, 96), device=DEV)
    bs.grouped_gemm_swiglu(s["xq"], 416, s["w1q"], 96, s["st"], R, probs=s["p"], y=y, y_dtype=bs.OUT_F32)
    for _ in range(20):
        z = torch.empty_like(y)
        s["xq"]["row_q"][T:].random_(0, 256)
        bs.grouped_gemm_swiglu(s["xq"], 416, s["w1q"], 96, s["st"], R, probs=s["p"], y=z, y_dtype=bs.OUT_F32)
        assert torch.equal(z[:T], y[:T])


def ragged(experts, rows, seed):
    """Sizes of `experts` groups with `rows` rows in all, about an eighth of them empty, one holding a tenth."""
    rng = np.random.default_rng(seed)
    w = rng.random(experts) * (rng.random(experts) > 0.125)
    w[experts // 2] = w.sum() / 9 + 1e-3
    k = np.floor(w / w.sum() * rows).astype(int)
    k[experts // 2] += rows - k.sum()
    return [int(v) for v in k]


# sizes that take each kernel: 128 x 128 tiles with long and short K steps (the second also with more groups than a
# wave's lanes), 256 x 256 tiles; each with K that ends inside a step and outputs that end inside a tile
LARGE = [(9, 2000, 160, 1056), (9, 2000, 1056, 1056), (70, 4100, 96, 1056), (70, 4100, 608, 1056), (64, 16400, 96, 4128),
         (40, 24000, 416, 4128)]


@pytest.mark.parametrize("experts,rows,hidden,ffn", LARGE)
def test_forward_in_tiles(experts, rows, hidden, ffn):
    flush(f"{experts} {rows} {hidden} {ffn}")
    s = operands(ragged(experts, rows, hidden), hidden, ffn, 31)
    R, T = s["R"], s["T"]
    ab = torch.full((R, 2 * ffn), float("nan"), dtype=torch.bfloat16, device=DEV)
    y = torch.full((R, ffn), float("nan"), device=DEV)
    out = poisoned(R, ffn, experts)
    bs.grouped_gemm_swiglu(s["xq"], hidden, s["w1q"], ffn, s["st"], R, probs=s["p"], ab=ab, y=y, y_dtype=bs.OUT_F32,
                           out=out)
    rab, tab, ry, ty = forward64(s)
    within(ab[:T], rab, 2.0 ** -8 * rab.abs() + 1.01 * tab, "ab")
    within(y[:T], ry, ty, "y")
    assert bool(ab[T:].isnan().all()) and bool(y[T:].isnan().all())
    check_exact_quantization(out, y, s)
    check_untouched(out, s, ffn)


@pytest.mark.parametrize("experts,rows,hidden,ffn", LARGE)
def test_gradient_in_tiles(experts, rows, hidden, ffn):
    flush(f"{experts} {rows} {hidden} {ffn}")
    s = operands(ragged(experts, rows, hidden + 1), hidden, ffn, 33)
    R, T = s["R"], s["T"]
    dab = torch.full((R, 2 * ffn), float("nan"), dtype=torch.bfloat16, device=DEV)
    dp = torch.full((R,), float("nan"), device=DEV)
    out = poisoned(R, 2 * ffn, experts)
    for _ in range(2):  # the second call finds its workspace and outputs used
        bs.grouped_gemm_swiglu_grad(s["xq"], hidden, s["w2q"], ffn, s["ab"], s["st"], R, probs=s["p"], dab=dab, out=out,
                                    dprobs=dp)
    rd, td, rp, tp = backward64(s)
    within(dab[:T], rd, 2.0 ** -8 * rd.abs() + 1.01 * td, "dab")
    within(dp[:T], rp, tp, "dprobs")
    assert bool(dab[T:].isnan().all()) and bool(dp[T:].isnan().all())
    check_close_quantization(out, rd, td, s)
    check_untouched(out, s, 2 * ffn)


@pytest.mark.parametrize("experts,rows", [(5, 30), (9, 2000), (70, 4100)])
def test_scales_at_their_ends(experts, rows):
    """Operand scale bytes from 0 (2^-127) up: rows whose values are subnormal or tiny, beside ordinary ones."""
    hidden, ffn = 160, 1056
    s = operands(ragged(experts, rows, 3), hidden, ffn, 35)
    T = s["T"]
    s["xq"]["row_s"][:, 0:T:3] = 0
    s["xq"]["row_s"][:, 1:T:3] = 1
    s["xv"] = deq(s["xq"]["row_q"][:T], s["xq"]["row_s"][:, :T])
    s["w1q"]["row_s"].view(-1)[:: 7] = 0
    s["w1v"] = deq(s["w1q"]["row_q"], s["w1q"]["row_s"]).view(experts, 2 * ffn, hidden)
    y = torch.empty((s["R"], ffn), device=DEV)
    bs.grouped_gemm_swiglu(s["xq"], hidden, s["w1q"], ffn, s["st"], s["R"], probs=s["p"], y=y, y_dtype=bs.OUT_F32)
    _, _, ry, ty = forward64(s)
    # values below bf16's and fp32's normal range may be flushed: 2^-126 of each of their products' other factors
    within(y[:T], ry, ty + 2.0 ** -100, "y")
