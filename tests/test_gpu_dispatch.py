"""Tokens to their experts and back: the plan against a loop on the host, the moved rows bit for bit, the quantized
rows against grouped_quantize of the same rows byte for byte, sums and gradients against 64 bits.

Tolerances.  A combined value is a chain of top_k fused multiply-adds and one addition in fp32, then one rounding: half a
step of the type times the value, and (top_k + 1) 2^-24 times the sum of its terms' sizes.  A weight's gradient is a sum of
cols products: chains of at most cols / 512 * 8 terms a lane, 6 lane steps and 8 waves."""
import numpy as np
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
MX, MX4 = bs.RECIPE_MX, bs.RECIPE_MX4


def choices_of(tokens, experts, k, seed=0, dropped=0.0, skew=0.0):
    rng = np.random.default_rng(seed)
    key = rng.random((tokens, max(experts, k))) + skew * np.arange(max(experts, k))
    e = np.argsort(-key, axis=1)[:, :k].astype(np.int32) % experts
    e[rng.random((tokens, k)) < dropped] = rng.choice([-1, experts, experts + 5, -7])
    return e, rng.random((tokens, k)).astype(np.float32)


def host_plan(e, probs, experts):
    flat = e.reshape(-1)
    order = [c for x in range(experts) for c in np.nonzero(flat == x)[0]] if experts < 64 else \
        [c for c in np.argsort(np.where((flat >= 0) & (flat < experts), flat, experts), kind="stable")
         if 0 <= flat[c] < experts]
    rows = np.full(flat.size, -1, np.int32)
    rows[order] = np.arange(len(order))
    choices = np.full(flat.size, -1, np.int32)
    choices[:len(order)] = order
    p = np.zeros(flat.size, np.float32)
    p[:len(order)] = probs.reshape(-1)[order]
    splits = np.array([(flat == x).sum() for x in range(experts)], np.int32)
    return splits, rows.reshape(e.shape), choices, p


def plan_of(e, experts, probs=None):
    return bs.dispatch_plan(torch.from_numpy(e).to(DEV), experts,
                            None if probs is None else torch.from_numpy(probs).to(DEV))


@pytest.mark.parametrize("tokens,experts,k,dropped,skew", [
    (1, 1, 1, 0, 0), (1, 8, 8, 0, 0), (4, 128, 8, 0, 0), (63, 5, 2, 0.3, 0), (64, 1024, 3, 0, 0), (65, 7, 1, 0, 3),
    (1023, 40, 4, 0, 0), (1024, 33, 4, 0.1, 0), (1025, 32, 4, 0, 1), (5000, 1024, 2, 0.5, 0), (9001, 128, 8, 0, 0.01),
    (40000, 3, 1, 1.0, 0), (70001, 256, 6, 0.2, 0)])
def test_plan(tokens, experts, k, dropped, skew):
    e, probs = choices_of(tokens, experts, k, 1, dropped, skew)
    got = plan_of(e, experts, probs)
    for name, want in zip(("splits", "rows", "choices", "probs"), host_plan(e, probs, experts)):
        assert np.array_equal(got[name].cpu().numpy(), want), name
    assert "probs" not in plan_of(e, experts)


def test_plan_of_large_chunks():
    """More than 512 units of choices: a workgroup takes several."""
    n, experts = (1 << 22) + 12345, 129
    g = torch.Generator(device=DEV).manual_seed(2)
    e = torch.randint(-1, experts + 1, (n, 1), generator=g, device=DEV, dtype=torch.int32)
    plan = bs.dispatch_plan(e, experts)
    bins = torch.where((e[:, 0] >= 0) & (e[:, 0] < experts), e[:, 0], experts)
    order = torch.sort(bins, stable=True).indices
    live = int((bins < experts).sum())
    assert torch.equal(plan["choices"][:live].long(), order[:live]) and (plan["choices"][live:] == -1).all()
    assert torch.equal(plan["splits"].long(), torch.bincount(bins, minlength=experts + 1)[:experts])
    rows = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    rows[order[:live]] = torch.arange(live, device=DEV, dtype=torch.int32)
    assert torch.equal(plan["rows"][:, 0], rows)


def test_plan_into_given_tensors_and_without_tokens():
    e, probs = choices_of(100, 9, 3, 3)
    want = plan_of(e, 9, probs)
    given = {k: torch.empty_like(v) for k, v in want.items()}
    got = bs.dispatch_plan(torch.from_numpy(e).to(DEV), 9, torch.from_numpy(probs).to(DEV), out=given)
    for k in want:
        assert got[k] is given[k] and torch.equal(got[k], want[k])
    none = bs.dispatch_plan(torch.empty((0, 3), dtype=torch.int32, device=DEV), 9)
    assert none["splits"].tolist() == [0] * 9 and none["choices"].numel() == 0
    assert bs.dispatch(torch.empty((0, 8), device=DEV), none).shape == (0, 8)
    assert bs.combine(torch.empty((0, 8), device=DEV), none).shape == (0, 8)
    assert bs.combine_grad(torch.empty((0, 8), device=DEV), none)["dy"].shape == (0, 8)


MOVES = [(1, 1, 1, 1), (3, 8, 2, 7), (5, 16, 3, 64), (4, 128, 8, 7168), (33, 6, 4, 130), (70, 9, 1, 2049),
         (300, 32, 6, 1000), (2, 1024, 32, 4100), (4500, 4, 2, 96), (5001, 7, 9, 515)]


def state(tokens, experts, k, cols, dtype, seed=4, dropped=0.2):
    e, probs = choices_of(tokens, experts, k, seed, dropped)
    plan = plan_of(e, experts)
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((tokens, cols), generator=g, device=DEV).to(dtype)
    y = torch.randn((tokens * k, cols), generator=g, device=DEV).to(dtype)
    live = int((plan["choices"] >= 0).sum())
    y[live:] = float("nan")  # rows past the last: not read
    return plan, x, y, torch.from_numpy(probs).to(DEV) - 0.25, live


@pytest.mark.parametrize("tokens,experts,k,cols", MOVES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("weighted", [False, True])
def test_dispatch(tokens, experts, k, cols, dtype, weighted):
    plan, x, _, w, live = state(tokens, experts, k, cols, dtype)
    x[0, 0] = float("nan")
    out = torch.full((tokens * k, cols), 77.0, dtype=dtype, device=DEV)
    got = bs.dispatch(x, plan, w if weighted else None, out=out)
    assert got is out and (out[live:] == 77).all()
    choices = plan["choices"][:live].long()
    want = x[choices // k]
    if weighted:
        want = (want.float() * w.view(-1)[choices][:, None]).to(dtype)
        assert torch.equal(torch.nan_to_num(out[:live]), torch.nan_to_num(want))
        assert torch.equal(out[:live].isnan(), want.isnan())
    else:
        bits = torch.int16 if dtype == torch.bfloat16 else torch.int32
        assert torch.equal(out[:live].view(bits), want.view(bits))


@pytest.mark.parametrize("tokens,experts,k,cols", MOVES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("weighted,added", [(False, False), (True, False), (True, True)])
def test_combine(tokens, experts, k, cols, dtype, weighted, added):
    plan, x, y, w, live = state(tokens, experts, k, cols, dtype)
    got = bs.combine(y, plan, w if weighted else None, x if added else None)
    choices = plan["choices"][:live].long()
    term = y[:live].double() * (w.view(-1)[choices].double()[:, None] if weighted else 1)
    ref, size = x.double() * added, x.double().abs() * added
    ref.index_add_(0, choices // k, term)
    size.index_add_(0, choices // k, term.abs())
    tol = HALF[dtype] * ref.abs() + (k + 1) * 2.0 ** -24 * 1.01 * size + 1e-45
    assert ((got.double() - ref).abs() <= tol).all()
    if added:  # in place
        same = bs.combine(y, plan, w, x, out=x)
        assert same is x and torch.equal(x, got)


@pytest.mark.parametrize("tokens,experts,k,cols", MOVES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_combine_grad(tokens, experts, k, cols, dtype):
    plan, dout, y, w, live = state(tokens, experts, k, cols, dtype)
    dy = torch.full((tokens * k, cols), 55.0, dtype=dtype, device=DEV)
    dw = torch.full((tokens, k), float("nan"), device=DEV)
    got = bs.combine_grad(dout, plan, y, w, dy=dy, dweights=dw)
    assert got["dy"] is dy and got["dweights"] is dw and (dy[live:] == 55).all()
    assert torch.equal(dy[:live], bs.dispatch(dout, plan, w)[:live])
    choices = plan["choices"][:live].long()
    prod = dout.double()[choices // k] * y[:live].double()
    ref = torch.zeros(tokens * k, dtype=torch.float64, device=DEV)
    size = ref.clone()
    ref[choices], size[choices] = prod.sum(1), prod.abs().sum(1)
    tol = ((cols / 512 + 1) * 8 + 14) * 2.0 ** -24 * size + 1e-45
    assert ((dw.view(-1).double() - ref).abs() <= tol).all()
    assert (dw.view(-1)[plan["rows"].view(-1) < 0] == 0).all()
    # either output alone, and dy over y
    assert torch.equal(bs.combine_grad(dout, plan, y, w, dy=False)["dweights"], dw)
    alone = bs.combine_grad(dout, plan, weights=w)
    assert "dweights" not in alone and torch.equal(alone["dy"][:live], dy[:live])
    over = bs.combine_grad(dout, plan, y, w, dy=y)
    assert torch.equal(over["dy"][:live], dy[:live]) and torch.equal(over["dweights"], dw)


def test_gradients_are_differences():
    """combine is linear in y and in the weights: its gradients by whole steps, in numbers that fp32 holds exactly."""
    e, _ = choices_of(6, 5, 3, 7, 0.3)
    plan = plan_of(e, 5)
    g = torch.Generator(device=DEV).manual_seed(7)
    ints = lambda *s: torch.randint(-4, 5, s, generator=g, device=DEV).float()  # noqa: E731
    y, w, dout = ints(18, 10), ints(6, 3), ints(6, 10)
    got = bs.combine_grad(dout, plan, y, w, dy=torch.zeros_like(y))
    base = (bs.combine(y, plan, w) * dout).sum()
    for t in range(6):
        for j in range(3):
            w2 = w.clone()
            w2[t, j] += 1
            assert (bs.combine(y, plan, w2) * dout).sum() - base == got["dweights"][t, j]
    for r in range(18):
        y2 = y.clone()
        y2[r, r % 10] += 1
        assert (bs.combine(y2, plan, w) * dout).sum() - base == got["dy"][r, r % 10]


QUANT = [(1, 1, 1, 32), (4, 128, 8, 7168), (40, 3, 2, 96), (129, 5, 1, 160), (300, 32, 6, 416), (1000, 7, 4, 128),
         (5, 1024, 32, 64), (2000, 2, 1, 1056)]


@pytest.mark.parametrize("tokens,experts,k,cols", QUANT)
@pytest.mark.parametrize("recipe", [MX, MX4])
@pytest.mark.parametrize("which", [bs.ROWWISE, bs.COLWISE, bs.ROWWISE | bs.COLWISE])
@pytest.mark.parametrize("dropped", [0.0, 0.3])
def test_dispatch_quantize_is_quantize_of_the_rows(tokens, experts, k, cols, recipe, which, dropped):
    plan, x, _, _, live = state(tokens, experts, k, cols, torch.bfloat16, 8, dropped)
    x[0, :32] = 0
    x[-1, -1] = 3e38
    n = tokens * k
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def poisoned():
        q = bs.alloc_quantized(n, cols, experts, recipe, which, DEV)
        for t in q.values():
            t.fill_(0xEE)
        return q

    got = bs.dispatch_quantize(x, plan, recipe, which, poisoned(), status=status)
    want = bs.grouped_quantize(bs.dispatch(x, plan, out=torch.zeros((n, cols), dtype=torch.bfloat16, device=DEV)),
                               plan["splits"], recipe, which, poisoned(), status=status)
    for name in want:
        assert torch.equal(got[name], want[name]), name
    assert int(status) == 0


@pytest.mark.parametrize("tokens,experts,k,cols", QUANT)
@pytest.mark.parametrize("recipe", [MX, MX4])
def test_weighted_dispatch_quantize(tokens, experts, k, cols, recipe):
    """Weights that are powers of two make bf16 products exact: the bytes of grouped_quantize again; and for any weights
    the rowwise MXFP8 values are within half a step of the fp32 products."""
    plan, x, _, w, live = state(tokens, experts, k, cols, torch.bfloat16, 9)
    n, both = tokens * k, bs.ROWWISE | bs.COLWISE
    two = torch.exp2(torch.randint(-3, 4, (tokens, k), device=DEV).float())
    got = bs.dispatch_quantize(x, plan, recipe, both, bs.alloc_quantized(n, cols, experts, recipe, both), weights=two)
    rows = bs.dispatch(x, plan, two)
    want = bs.grouped_quantize(rows, plan["splits"], recipe, both, bs.alloc_quantized(n, cols, experts, recipe, both))
    assert torch.equal(got["row_q"][:live], want["row_q"][:live])
    assert torch.equal(got["row_s"][:, :live], want["row_s"][:, :live])
    used = int(((plan["splits"].long() + 127) // 128 * 128).sum())
    per = 2 if recipe == MX4 else 1
    assert torch.equal(got["col_q"][:used * cols // per], want["col_q"][:used * cols // per])
    assert torch.equal(got["col_s"][:used * cols // 32], want["col_s"][:used * cols // 32])
    if recipe == MX:
        q = bs.dispatch_quantize(x, plan, MX, bs.ROWWISE, bs.alloc_quantized(n, cols, experts, MX, bs.ROWWISE), weights=w)
        c = plan["choices"][:live].long()
        v = x[c // k].float() * w.view(-1)[c][:, None]
        s = torch.exp2(q["row_s"][:, :live].t().double() - 127).repeat_interleave(32, 1)
        off = (q["row_q"][:live].view(torch.float8_e4m3fn).double() * s - v.double()).abs()
        assert (off <= 2.0 ** -4 * v.double().abs() + 2.0 ** -10 * s).all()
        top = v.view(live, -1, 32).abs().amax(2).double()
        s = s[:, ::32]
        assert (top <= 448 * s).all() and ((top > 224 * s) | (top == 0)).all()


def test_bad_sizes_set_the_status_and_write_nothing():
    e, _ = choices_of(64, 4, 2, 10)
    plan = plan_of(e, 4)
    x = torch.ones((64, 64), dtype=torch.bfloat16, device=DEV)
    for bad, bit in ((-1, bs.STATUS_NEGATIVE_SPLIT), (1000, bs.STATUS_EXCEEDS_CAPACITY)):
        plan["splits"][1] = bad
        q = bs.alloc_quantized(128, 64, 4, MX, bs.ROWWISE | bs.COLWISE)
        for t in q.values():
            t.fill_(0xEE)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        bs.dispatch_quantize(x, plan, MX, bs.ROWWISE | bs.COLWISE, q, status=status)
        assert int(status) == bit and all((t == 0xEE).all() for t in q.values())


def test_rows_that_a_plan_does_not_write_are_skipped():
    """Rows and choices outside their buffers are neither read nor written."""
    rows = torch.tensor([[0, 99], [-5, 3], [1 << 30, 1]], dtype=torch.int32, device=DEV)
    plan = {"rows": rows, "choices": torch.tensor([0, 5, 77, 3, -9, 1 << 30], dtype=torch.int32, device=DEV),
            "splits": torch.tensor([4], dtype=torch.int32, device=DEV)}
    x = torch.arange(3 * 32, device=DEV).view(3, 32).bfloat16()
    out = torch.full((6, 32), -1.0, dtype=torch.bfloat16, device=DEV)
    bs.dispatch(x, plan, out=out)
    assert torch.equal(out[0], x[0]) and torch.equal(out[3], x[1]) and torch.equal(out[1], x[2])
    assert (out[[2, 4, 5]] == -1).all()
    back = bs.combine(out, plan)
    assert torch.equal(back, torch.stack([out[0], out[3], out[1]]))
    q = bs.dispatch_quantize(x, plan, MX, bs.ROWWISE | bs.COLWISE, bs.alloc_quantized(6, 32, 1, MX, 3))
    assert (q["row_q"][2] == 0).all()


def test_streams_and_repeats_give_the_same_bits():
    plan, x, y, w, live = state(3000, 16, 4, 520, torch.bfloat16, 11)
    want = bs.combine(y, plan, w), bs.combine_grad(x, plan, y, w, dy=False)["dweights"]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, side, side.cuda_stream):
        got = bs.combine(y, plan, w, stream=stream), bs.combine_grad(x, plan, y, w, dy=False, stream=stream)["dweights"]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
