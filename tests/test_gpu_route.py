"""The router against its formulas in 64 bits: the choice as whole numbers, probabilities, sums and gradients within
what their fp32 operations can be off.

Tolerances.  A score is a few fp32 operations on an exponential: expf is within 2 ulp, its argument l - m off by half an
ulp of up to |l - m| < 32 (relative 2^-20 of the result); the stated sigmoid's exp2s is within 3e-7 at an argument off by
2 half-ulps of up to 46.  2^-17 relative covers both with their sums over up to 1024 experts (chains of 16 a lane and 6
lane steps: 22 * 2^-24) and divisions.  Logits are drawn within +-16."""
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

pytestmark = pytest.mark.gpu
DEV = "cuda"
REL = 2.0 ** -17
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
SOFTMAX, SIGMOID = bs.ROUTE_SOFTMAX, bs.ROUTE_SIGMOID


def draw(tokens, experts, dtype, seed=0, masked=0.0, scale=2.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    l = (torch.randn((tokens, experts), generator=g, device=DEV) * scale).clamp(-16, 16)
    if masked:
        l[torch.rand((tokens, experts), generator=g, device=DEV) < masked] = -torch.inf
    bias = torch.randn(experts, generator=g, device=DEV) * 0.2
    return l.to(dtype), bias, g


def exp2s(x):
    """The stated 2^x, by numpy in fp32 (one rounding per operation)."""
    import numpy as np
    f = np.float32
    x = np.clip(x, f(-126), f(126))
    k = np.floor(x + f(0.5))
    r = x - k
    p = np.full_like(x, f(1.52527338e-05))
    for c in (0.000154035304, 0.00133335581, 0.00961812911, 0.0555041087, 0.240226507, 0.693147182, 1.0):
        p = p * r + f(c)
    return np.ldexp(p, k.astype(np.int32))


def keys_of(l, bias, scoring):
    """The keys in fp32, by their statement, on the host."""
    import numpy as np
    x = l.float().cpu().numpy()
    if scoring == SIGMOID:
        with np.errstate(all="ignore"):
            key = np.float32(1) / (np.float32(1) + exp2s(-x * np.float32(1.44269502)))
    else:
        key = x
    if bias is not None:
        key = key + bias.cpu().numpy()[None, :]
    return np.where(np.isneginf(x), np.float32(-np.inf), key)


def choose(key, k):
    import numpy as np
    order = np.argsort(-key, axis=1, kind="stable")[:, :k]
    return np.where(np.isneginf(np.take_along_axis(key, order, 1)), -1, order)


def probs64(l, experts, scoring, renormalize, scale):
    """(probs, score_sum) in 64 bits, differentiable in l."""
    open_ = ~torch.isneginf(l)
    safe = torch.where(open_, l, 0.0)
    if scoring == SOFTMAX:
        top = torch.where(open_, safe.detach(), -1e30).amax(1, keepdim=True)
        w = torch.where(open_, torch.exp(safe - top), 0.0)
        s = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        s = torch.where(open_, torch.sigmoid(safe), 0.0)
    p = torch.where(experts >= 0, s.gather(1, experts.long().clamp(min=0)), 0.0)
    if renormalize:
        p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
    return p * scale, s.sum(0)


SHAPES = [(1, 1, 1), (1, 8, 2), (3, 17, 3), (5, 16, 16), (4, 128, 8), (67, 33, 4), (9, 256, 8), (7, 257, 6), (6, 512, 20),
          (5, 1024, 32), (1000, 64, 6), (4099, 130, 5)]


@pytest.mark.parametrize("tokens,experts,k", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scoring,renormalize,biased", [(SOFTMAX, True, False), (SOFTMAX, False, True),
                                                        (SIGMOID, True, True), (SIGMOID, False, False)])
@pytest.mark.parametrize("masked", [0.0, 0.4])
def test_forward(tokens, experts, k, dtype, scoring, renormalize, biased, masked):
    l, bias, _ = draw(tokens, experts, dtype, 1, masked)
    if masked and tokens > 2:
        l[1] = -torch.inf  # a token without any expert
    bias = bias if biased else None
    total = torch.full((experts,), float("nan"), device=DEV)
    got = bs.route_topk(l, k, scoring, bias, renormalize, 2.5, score_sum=total)
    want = choose(keys_of(l, bias, scoring), k)
    assert (got["experts"].cpu().numpy() == want).all()
    p, s = probs64(l.double(), got["experts"], scoring, renormalize, 2.5)
    assert ((got["probs"] - p).abs() <= REL * p).all()
    assert (got["probs"][got["experts"] < 0] == 0).all()
    # a sum over tokens: chains of at most tokens / blocks and 1024 / 16 blocks, 16 groups and 16 waves
    blocks = bs.route_topk_workspace_bytes(tokens, experts) // (4 * experts)
    assert ((total - s).abs() <= (REL + (tokens / blocks + blocks / 16 + 40) * 2.0 ** -24) * s).all()


def test_ties_take_the_lowest_index():
    for experts in (40, 300):
        l = torch.zeros((6, experts), device=DEV)
        l[1] = torch.tensor([1.0, 2.0] * (experts // 2), device=DEV)
        l[2, ::3] = -0.0
        l[3, 7:] = 5.0
        l[4, 3] = torch.nan
        l[4, 9] = torch.inf
        l[4, 30] = -torch.nan
        l[5] = -torch.inf
        l[5, 11] = -3.4e38
        e = bs.route_topk(l, 4)["experts"].tolist()
        assert e == [[0, 1, 2, 3], [1, 3, 5, 7], [0, 1, 2, 3], [7, 8, 9, 10], [3, 30, 9, 0], [11, -1, -1, -1]]


def test_bias_of_minus_infinity_masks():
    l, bias, _ = draw(50, 20, torch.float32)
    bias[4] = -torch.inf
    for scoring in (SOFTMAX, SIGMOID):
        got = bs.route_topk(l, 20, scoring, bias)
        assert not (got["experts"] == 4).any() and (got["experts"][:, -1] == -1).all()
        assert (got["experts"][:, :-1] >= 0).all()


@pytest.mark.parametrize("extreme", [60.0, 1e4])
def test_far_logits(extreme):
    """Scores that underflow: the renormalized probabilities of the chosen still sum to scale."""
    l = torch.zeros((2, 64), device=DEV)
    l[:, 5] = extreme
    bias = torch.zeros(64, device=DEV)
    bias[:5] = 2 * extreme  # the choice avoids the largest logit
    got = bs.route_topk(l, 4, SOFTMAX, bias)
    assert got["experts"].tolist() == [[0, 1, 2, 3]] * 2
    assert torch.equal(got["probs"], torch.full((2, 4), 0.25, device=DEV))
    low = bs.route_topk(torch.full((2, 64), -extreme, device=DEV), 4, SIGMOID)
    assert torch.equal(low["probs"], torch.full((2, 4), 0.25, device=DEV))


@pytest.mark.parametrize("tokens,experts,k", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scoring", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renormalize,summed,masked", [(True, False, 0.4), (True, True, 0.0), (False, True, 0.4),
                                                       (False, False, 0.0)])
def test_gradient(tokens, experts, k, dtype, scoring, renormalize, summed, masked):
    l, bias, g = draw(tokens, experts, dtype, 2, masked)
    if masked and tokens > 2:
        l[1] = -torch.inf
    e = bs.route_topk(l, k, scoring, bias, renormalize, 1.5)["experts"]
    dp = torch.randn((tokens, k), generator=g, device=DEV)
    ds = torch.randn(experts, generator=g, device=DEV) if summed else None
    got = bs.route_topk_grad(dp, l, e, scoring, renormalize, 1.5, ds)
    assert got.dtype == dtype
    x = l.double().requires_grad_()
    p, s = probs64(x, e, scoring, renormalize, 1.5)
    loss = (p * dp.double()).sum() + (0 if ds is None else (s * ds.double()).sum())
    loss.backward()
    # a term of a logit's gradient is at most its score (chosen over their sum) times the token's largest |dp| or |ds|
    with torch.no_grad():
        part, _ = probs64(l.double(), e, scoring, renormalize, 1.5)
        size = torch.zeros_like(x).scatter_add_(1, e.long().clamp(min=0), part) * dp.abs().amax(1, keepdim=True)
        full, _ = probs64(l.double(), torch.arange(experts, device=DEV).expand(tokens, -1), scoring, False, 1.5)
        size += full * ((0 if ds is None else ds.abs().max()) + (0 if renormalize else dp.abs().amax(1, keepdim=True)))
    # (the reference's own rounding, where the formula's terms cancel to 0 as they do for logits that are not chosen:
    # at most 1024 + 32 double operations, each off by 2^-53 of terms of at most 1.5 |dp| or |ds|: below 2^-41)
    most = dp.abs().max() + (0 if ds is None else ds.abs().max())
    tol = HALF[dtype] * x.grad.abs() + 4 * REL * size + 2.0 ** -41 * most
    assert ((got - x.grad).abs() <= tol).all()
    assert (got[torch.isneginf(l)] == 0).all()


@pytest.mark.parametrize("scoring,renormalize", [(SOFTMAX, True), (SOFTMAX, False), (SIGMOID, True), (SIGMOID, False)])
def test_gradient_is_the_forwards_differences(scoring, renormalize):
    """Central differences of the kernel's own forward, in steps that the choice survives."""
    l, _, g = draw(3, 24, torch.float32, 3)
    dp, ds = torch.randn((3, 5), generator=g, device=DEV), torch.randn(24, generator=g, device=DEV)
    base = bs.route_topk(l, 5, scoring, None, renormalize)
    grad = bs.route_topk_grad(dp, l, base["experts"], scoring, renormalize, 1.0, ds)
    h = 2.0 ** -6
    for t, e in [(0, int(base["experts"][0, 1])), (1, int(base["experts"][1, 4])), (2, 0), (0, 23)]:
        loss = []
        for sign in (1, -1):
            x = l.clone()
            x[t, e] += sign * h
            total = torch.empty(24, device=DEV)
            r = bs.route_topk(x, 5, scoring, None, renormalize, score_sum=total)
            if not torch.equal(r["experts"], base["experts"]):
                pytest.skip("the choice changes within the step")
            loss.append(float((r["probs"].double() * dp).sum() + (total.double() * ds).sum()))
        # third derivatives of a sigmoid or a softmax are below 1/4 (times |dp| and |ds| below 4 at 6 terms)
        assert abs((loss[0] - loss[1]) / (2 * h) - float(grad[t, e])) < 6 * h * h + 1e-4


def test_an_expert_that_stands_twice():
    l, _, g = draw(9, 12, torch.float32, 4)
    e = torch.randint(-2, 14, (9, 6), generator=g, device=DEV, dtype=torch.int32)
    dp = torch.randn((9, 6), generator=g, device=DEV)
    for scoring in (SOFTMAX, SIGMOID):
        for renormalize in (True, False):
            got = bs.route_topk_grad(dp, l, e, scoring, renormalize)
            x = l.double().requires_grad_()
            p, _ = probs64(x, torch.where(e < 12, e, -1), scoring, renormalize, 1.0)
            (p * dp.double()).sum().backward()
            assert ((got - x.grad).abs() <= 64 * REL * dp.abs().max()).all()


def test_given_outputs_no_tokens_and_other_streams():
    l, bias, _ = draw(300, 64, torch.bfloat16, 5)
    total = torch.empty(64, device=DEV)
    want = bs.route_topk(l, 4, SIGMOID, bias, score_sum=total)
    want = {k: v.clone() for k, v in want.items()}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream, None):
        given = dict(probs=torch.empty(300, 4, device=DEV), experts=torch.empty((300, 4), dtype=torch.int32, device=DEV),
                     score_sum=torch.empty(64, device=DEV))
        torch.cuda.synchronize()
        got = bs.route_topk(l, 4, SIGMOID, bias, stream=stream, **given)
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(got[k], want[k]) and got[k] is given[k]
    empty = bs.route_topk(l[:0], 4, score_sum=total)
    assert empty["probs"].shape == (0, 4) and (total == 0).all()
    assert bs.route_topk_grad(empty["probs"], l[:0], empty["experts"]).shape == (0, 64)
