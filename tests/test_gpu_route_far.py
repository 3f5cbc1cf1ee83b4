"""Scores of logits far below a token's largest: as exact as those next to it.

Tolerance.  The logits are multiples of 2^-8 below 2^7, so that their differences x are exact, and the score's error is, in
units of 2^-24, that of the exponential (the hardware's 2^y: 1 ulp, 2; what y = x log2(e) was rounded by is made good but
for the rounding of ln 2, 2.7e-9 |x|: 3.7 at 80; the last step 0.5), that of the sum (its terms' 6.2, chains of at most 16 a
lane and 6 lane steps: 22), its reciprocal and a product (0.5 each): below 36.  Without making good y's rounding: 44 at 80 from
half an ulp of y, and 12 from that of log2(e), more."""
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

pytestmark = pytest.mark.gpu
DEV = "cuda"
REL = 36 * 2.0 ** -24


def draw(tokens, experts, dtype, seed):
    """Logits from -60 to 0, and one expert a token on top."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    step = 2.0 ** -8 if dtype == torch.float32 else 0.5
    l = -torch.randint(0, int(60 / step) + 1, (tokens, experts), generator=g, device=DEV).float() * step
    l[torch.arange(tokens), torch.randint(0, experts, (tokens,), generator=g, device=DEV)] = 20.0
    return l.to(dtype)


def scores64(l):
    return torch.softmax(l.double(), 1)


@pytest.mark.parametrize("experts", [7, 16, 64, 128, 256, 300, 1024])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_tokens_scores(experts, dtype):
    """The sums over one token are its scores."""
    for seed in range(5):
        l = draw(1, experts, dtype, seed)
        total = torch.empty(experts, device=DEV)
        bs.route_topk(l, 1, score_sum=total)
        want = scores64(l)[0]
        assert ((total - want).abs() <= REL * want).all(), float(((total - want).abs() / want).max() * 2 ** 24)


@pytest.mark.parametrize("experts,k", [(7, 7), (64, 32), (128, 32), (300, 32), (1024, 20)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_probabilities_as_they_are(experts, k, dtype):
    """Half of the experts are chosen before the other half, whatever their scores."""
    l = draw(500, experts, dtype, 1)
    bias = torch.zeros(experts, device=DEV)
    bias[::2] = 300.0
    got = bs.route_topk(l, k, bias=bias, renormalize=False)
    want = scores64(l).gather(1, got["experts"].long())
    assert ((got["probs"] - want).abs() <= REL * want).all(), float(((got["probs"] - want).abs() / want).max() * 2 ** 24)


@pytest.mark.parametrize("experts", [16, 128, 300])
def test_gradient_of_the_scores(experts):
    """d = s (g - sum g s): with g = 1 at every other expert and the largest's 0, the small scores' gradients are theirs."""
    l = draw(300, experts, torch.float32, 2)
    s = scores64(l)
    ds = torch.zeros(experts, device=DEV)
    ds[::2] = 1.0
    e = torch.full((300, 1), -1, dtype=torch.int32, device=DEV)
    got = bs.route_topk_grad(torch.zeros((300, 1), device=DEV), l, e, dscore_sum=ds)
    mean = (s * ds).sum(1, keepdim=True)
    # (the mean by as long chains, and a subtraction and a product more)
    assert ((got - s * (ds - mean)).abs() <= (2 * REL + 2.0 ** -22) * s).all()


def test_masked_and_undefined_logits():
    l = draw(6, 40, torch.float32, 3)
    l[0, 5:] = -torch.inf
    l[1] = -torch.inf
    l[2, 4] = torch.nan
    l[3, 7] = -3.4e38
    total = torch.empty(40, device=DEV)
    for t in range(6):
        bs.route_topk(l[t:t + 1], 4, score_sum=total)
        want = scores64(l[t:t + 1])[0] if t != 1 else torch.zeros(40, device=DEV, dtype=torch.float64)
        assert torch.equal(total.isnan(), want.isnan())
        assert (total.isnan() | ((total - want).abs() <= REL * want + 2.0 ** -126)).all()
