"""Stochastic rounding of AdamW's 8-bit states: where they go, how often, and what that does over many steps.

Tolerances.  A stored state lies within one e4m3 step of the unrounded one: 2^-3 of its power of two, or 2^-9 of the
block's scale; the fp32 arithmetic before it is off by 8 * 2^-24 of its terms.  A mean of n roundings, each off by at
most one step with a variance of at most a quarter, is within 5 / (2 sqrt(n)) steps of its expectation (5 standard
deviations), besides the 2^-17 by which the 16 random bits' probabilities are off."""
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = torch.float8_e4m3fn
U = 2.0 ** -24


def state(n, seed, spread=0.0):
    """One tensor of n elements with 8-bit states; spread: the gradients' and states' size varies by exp(spread * randn)."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    nb, size = (n + 127) // 128, torch.exp(spread * rand(n))
    return dict(p=rand(n) * 0.05, g=rand(n) * 1e-2 * size,
                m=(rand(n) * 60 * size).clamp(-448, 448).to(E4M3).view(torch.uint8),
                v=(rand(n).abs() * 60 * size).clamp(max=448).to(E4M3).view(torch.uint8),
                ms=rand(nb).abs() * 1e-4 + 1e-5, vs=rand(nb).abs() * 1e-4 + 1e-5)


def plan_of(s, **more):
    return bs.adamw_plan([s["p"]], [s["g"]], [s["m"]], [s["v"]], [s["ms"]], [s["vs"]], **more)


def clone(s):
    return {k: t.clone() for k, t in s.items()}


def value(code, scale):
    return code.view(E4M3).double() * scale.double().repeat_interleave(128)[:code.numel()]


def spacing(x, scale):
    """The e4m3 step around x > 0 in a block of this scale."""
    e = torch.frexp((x / scale).clamp(min=2.0 ** -6))[1] - 1
    return scale * torch.exp2((e - 3).double())


@pytest.mark.parametrize("spread", [0.0, 3.0])
def test_states_go_to_a_neighbour_without_bias(spread):
    n, b1, b2 = 1 << 20, 0.9, 0.95
    s = state(n, 1, spread)
    g, m, u = s["g"].double(), value(s["m"], s["ms"]), value(s["v"], s["vs"])
    terms = b1 * m.abs() + (1 - b1) * g.abs()
    m, u = b1 * m + (1 - b1) * g, (b2 * u * u + (1 - b2) * g * g).sqrt()
    near = clone(s)
    bs.adamw_step(plan_of(near), 1e-3, b1, b2, step=4)
    bs.adamw_step(plan_of(s), 1e-3, b1, b2, step=4, seed=17)
    for k in ("p", "ms", "vs"):  # these do not depend on how the states are rounded
        assert torch.equal(s[k], near[k]), k
    for code, scale, x, size, low in ((s["m"], s["ms"], m, terms, 0.0), (s["v"], s["vs"], u, u, 2.0 ** -9)):
        wide = scale.double().repeat_interleave(128)[:n]
        keep = x.abs() >= low * wide  # (below its smallest code a second state is not rounded up and down evenly)
        code, x, wide, size = code[keep], x[keep], wide[keep], size[keep]
        got, one = code.view(E4M3).double() * wide, spacing(x.abs(), wide)
        off = (got - x) / one
        assert bool((off.abs() <= 1 + 2.0 ** -16 + 8 * U * size / one).all())
        assert abs(float((off * x.sign()).mean())) <= 2.5 / x.numel() ** 0.5 + 2.0 ** -17 + 1e-4
        # in the subnormal codes by themselves, and by how far up a step the value lies
        at = (x.abs() / one) % 1
        small = x.abs() / wide < 2.0 ** -6
        assert spread == 0.0 or int(small.sum()) > 10000
        for where in [small] + [(~small) & (at >= q / 8) & (at < (q + 1) / 8) for q in range(8)]:
            c = int(where.sum())
            if c > 1000:
                assert abs(float((off * x.sign())[where].mean())) <= 2.5 / c ** 0.5 + 2.0 ** -17 + 1e-4


def test_same_arguments_same_bits():
    def run(seed, step):
        s = state(5000, 2)
        bs.adamw_step(plan_of(s), 1e-3, step=step, seed=seed)
        return s

    a, b = run(5, 3), run(5, 3)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    for other in (run(6, 3), run(5 + (1 << 32), 3), run(-5, 3)):
        assert not torch.equal(a["m"], other["m"]) and not torch.equal(a["v"], other["v"])
    # two tensors of a plan, and two blocks of one, do not share their bits
    x = [state(4096, 3) for _ in range(2)]
    for s in x:
        for k in ("p", "g", "m", "v"):
            s[k][128:] = s[k][:128].repeat(31)
        s["ms"].fill_(1e-4), s["vs"].fill_(1e-4)
    bs.adamw_step(bs.adamw_plan(*[[s[k] for s in x] for k in ("p", "g", "m", "v", "ms", "vs")]), 1e-3, step=2, seed=9)
    assert not torch.equal(x[0]["m"], x[1]["m"]) and not torch.equal(x[0]["v"], x[1]["v"])
    for k in ("m", "v"):
        rows = x[0][k].view(-1, 128)
        assert len(torch.unique(rows, dim=0)) == len(rows)


def test_a_state_that_is_a_code_stays():
    """beta1 = beta2 = 0: the states are the gradients; those that are codes of the block's scale come back exactly."""
    n = 1024
    s = state(n, 4)
    codes = torch.arange(1, 127, dtype=torch.uint8, device=DEV)
    for b in range(n // 128):  # every positive code, 448 among them, in each block; two zeros
        s["g"][128 * b:128 * b + 126] = codes.view(E4M3).float() * 2.0 ** -10
        s["g"][128 * b + 126:128 * b + 128] = 0
    sf = torch.tensor(448 * 2.0 ** -10, dtype=torch.float32, device=DEV) * torch.tensor(1 / 448, dtype=torch.float32)
    assert float(sf) == 2.0 ** -10  # (so that the division by it is exact)
    bs.adamw_step(plan_of(s), 1e-3, 0.0, 0.0, step=1, seed=3)
    want = torch.cat([codes, codes.new_zeros(2)]).repeat(n // 128)
    assert torch.equal(s["m"], want) and torch.equal(s["v"], want)


def test_graph_with_device_step():
    s = state(6000, 5)
    e = clone(s)
    plan, eager = plan_of(s), plan_of(e)
    step = torch.ones(1, dtype=torch.int32, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bs.adamw_step(plan, 1e-3, step_dev=step, seed=11)
    for t in range(1, 5):
        step.fill_(t)
        s["g"].copy_(torch.randn_like(s["g"]))
        e["g"].copy_(s["g"])
        graph.replay()
        torch.cuda.synchronize()
        bs.adamw_step(eager, 1e-3, step=t, seed=11)
        for k in s:
            assert torch.equal(s[k], e[k]), (t, k)


def test_fp32_states_do_not_depend_on_the_seed():
    g = torch.Generator(device=DEV).manual_seed(1)
    a = [torch.randn(777, generator=g, device=DEV) for _ in range(3)] + [torch.rand(777, generator=g, device=DEV)]
    b = [t.clone() for t in a]
    bs.adamw_step(bs.adamw_plan(*[[t] for t in a]), 1e-3, step=2)
    bs.adamw_step(bs.adamw_plan(*[[t] for t in b]), 1e-3, step=2, seed=4)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def follow(beta2, gradients, blocks=64):
    """Runs the gradients [step] -> (the block's first element's, the others') on fp32 and on 8-bit states; returns what
    the others' sqrt(v) and updates are at the end: fp32's value, and the 8-bit ones' means."""
    n, lr = 128 * blocks, 1e-3
    s = dict(p=torch.zeros(n, device=DEV), g=torch.zeros(n, device=DEV), m=torch.zeros(n, dtype=torch.uint8, device=DEV),
             v=torch.zeros(n, dtype=torch.uint8, device=DEV), ms=torch.zeros(blocks, device=DEV),
             vs=torch.zeros(blocks, device=DEV))
    plan = plan_of(s)
    f = [torch.zeros(n, device=DEV) for _ in range(4)]
    f[1] = s["g"]
    plain = bs.adamw_plan(*[[t] for t in (f[0], f[1], f[2], f[3])])
    wide = s["g"].view(blocks, 128)
    for t, (first, others) in enumerate(gradients, 1):
        wide[:, 0], wide[:, 1:] = first, others
        if t == len(gradients):
            s["p"].zero_(), f[0].zero_()
        bs.adamw_step(plan, lr, 0.9, beta2, 1e-8, 0.0, t, seed=7)
        bs.adamw_step(plain, lr, 0.9, beta2, 1e-8, 0.0, t)
    keep = torch.ones(n, dtype=torch.bool, device=DEV).view(blocks, 128)
    keep[:, 0] = False
    keep = keep.view(-1)
    u, upd = value(s["v"], s["vs"])[keep], s["p"].double()[keep] / lr
    return float(f[3].sqrt()[1]), float(f[0][1] / lr), u, upd


# A code's step is at most 2^-3 of its value: the state of a single element strays by some such steps from the unrounded
# one, the mean over 8128 elements stays within one.
@pytest.mark.parametrize("beta2,steps", [(0.95, 400), (0.999, 12000)])
@pytest.mark.parametrize("low,high", [(0.01, 1.0), (1.0, 0.01)])
def test_second_state_follows_gradients_that_fall_and_rise(beta2, steps, low, high):
    """One element's gradient stays at 1 and holds the block's scale; the others' change by a factor of 100."""
    if low > high:
        steps = steps // 4  # (a rise shows after some 1 / (1 - beta2) steps)
    grads = [(1.0, high)] * 200 + [(1.0, low)] * steps
    want, upd32, u, upd = follow(beta2, grads)
    assert abs(float(u.mean()) / want - 1) < 0.125, (float(u.mean()), want)
    assert abs(float(upd.mean()) / upd32 - 1) < 0.25, (float(upd.mean()), upd32)


def test_states_vanish_when_gradients_stop():
    """Rounded to nearest, the lowest codes of m stay for ever and move their parameters at every step."""
    want, upd32, u, upd = follow(0.999, [(1.0, 1e-4)] * 100 + [(1.0, 0.0)] * 500)
    assert abs(upd32) < 1e-15 and not bool(upd.any())


def test_training_follows_fp32_states():
    """The default beta2 on a quadratic whose gradients span four decades inside every block."""
    n, loss = 4096, []
    g = torch.Generator(device=DEV).manual_seed(2)
    width = 10.0 ** (-4 * torch.rand(n, generator=g, device=DEV))
    target = torch.randn(n, generator=g, device=DEV)
    for q8 in (False, True):
        s = dict(p=torch.zeros(n, device=DEV), g=torch.zeros(n, device=DEV))
        z = [torch.zeros(n, dtype=torch.uint8 if q8 else torch.float32, device=DEV) for _ in range(2)]
        sc = [[torch.zeros(n // 128, device=DEV)] for _ in range(2)] if q8 else [None, None]
        plan = bs.adamw_plan([s["p"]], [s["g"]], [z[0]], [z[1]], *sc)
        noise = torch.Generator(device=DEV).manual_seed(3)
        for t in range(1, 1001):
            s["g"].copy_(width * (s["p"] - target + 0.1 * torch.randn(n, generator=noise, device=DEV)))
            bs.adamw_step(plan, 1e-2, step=t, weight_decay=0.0, seed=1)
        loss.append(float((s["p"] - target).square().mean()))
    assert loss[0] < 0.05 and loss[1] < 2 * loss[0] + 0.01, loss
