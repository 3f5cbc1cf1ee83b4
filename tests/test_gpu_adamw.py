"""The AdamW step against its formulas in 64 bits.

Tolerances.  m and v are three and four fp32 roundings of terms of one sign pattern: 4 * 2^-24 of
their terms' sizes; p's update is m / (sqrt(v) root + eps) step_size, whose relative error is the
sum of its factors' (m's terms over m counted in full, at most 12 roundings), and p is rounded once
more (bf16 2^-8, fp32 2^-24).  An 8-bit state is half a step of e4m3 off: 2^-4 of its value, or half
of the smallest step, 2^-10 of its block's scale; the scale is amax / 448 to 8 * 2^-24."""
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
E4M3 = torch.float8_e4m3fn


def tensors(sizes, pt, gt, q8, copy, seed=0, shift=0):
    """Lists of tensors; with `shift`, each begins that many elements into its own allocation."""
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rand(n, scale):
        return torch.randn(n, generator=g, device=DEV) * scale

    def place(v):
        b = torch.empty(v.numel() + shift, dtype=v.dtype, device=DEV)
        b[shift:] = v
        return b[shift:]

    s = dict(p=[place(rand(n, 0.05).to(pt)) for n in sizes], g=[place(rand(n, 1e-2).to(gt)) for n in sizes])
    if q8:
        nb = [(n + 127) // 128 for n in sizes]
        s["m"] = [place(rand(n, 60).clamp(-448, 448).to(E4M3).view(torch.uint8)) for n in sizes]
        s["v"] = [place(rand(n, 60).abs().clamp(max=448).to(E4M3).view(torch.uint8)) for n in sizes]
        s["ms"] = [rand(n, 1).abs() * 1e-4 for n in nb]
        s["vs"] = [rand(n, 1).abs() * 1e-4 for n in nb]
    else:
        s["m"], s["v"] = [place(rand(n, 5e-3)) for n in sizes], [place(rand(n, 1e-2).square()) for n in sizes]
        s["ms"] = s["vs"] = None
    s["c"] = [place(torch.zeros(n, dtype=torch.bfloat16, device=DEV)) for n in sizes] if copy else None
    return s


def plan_of(s, **more):
    return bs.adamw_plan(s["p"], s["g"], s["m"], s["v"], s["ms"], s["vs"], s["c"], **more)


def states64(s, i):
    if s["ms"] is None:
        return s["m"][i].double(), s["v"][i].double()
    n = s["p"][i].numel()
    m = s["m"][i].view(E4M3).double() * s["ms"][i].double().repeat_interleave(128)[:n]
    u = s["v"][i].view(E4M3).double() * s["vs"][i].double().repeat_interleave(128)[:n]
    return m, u * u


def step64(p, g, m, v, step, gs=1.0, lr=0, beta1=0, beta2=0, eps=0, weight_decay=0):
    """New p, m, v in 64 bits, the size of m's terms, and the size of the update's."""
    g = g * gs
    size = (beta1 * m).abs() + ((1 - beta1) * g).abs()
    m, v = beta1 * m + (1 - beta1) * g, beta2 * v + (1 - beta2) * g * g
    by = (v / (1 - beta2 ** step)).sqrt() + eps
    k = lr / (1 - beta1 ** step)
    return p - lr * weight_decay * p - k * m / by, m, v, size, k * size / by


def within(got, ref, tol, what):
    err = (got.double() - ref).abs()
    assert bool((err <= tol + 1e-35).all()), f"{what}: {float((err / (tol + 1e-35)).max()):.3g} times the bound"


def check_step(s, before, i, ref, what=""):
    p, m, v, size, upd = ref
    pt = s["p"][i].dtype
    old = before["p"][i].double().abs()
    within(s["p"][i], p, HALF[pt] * p.abs() + U * (4 * old + 16 * upd), f"{what} p")
    if s["c"] is not None:
        within(s["c"][i], p, 2.0 ** -8 * p.abs() * (1 + 2.0 ** -7) + U * (4 * old + 16 * upd), f"{what} copy")
    if s["ms"] is None:
        within(s["m"][i], m, 4 * U * size, f"{what} m")
        within(s["v"][i], v, 6 * U * v, f"{what} v")
        return
    for name, x, terms in (("m", m, size), ("v", v.sqrt(), v.sqrt())):
        n = x.numel()
        nb = (n + 127) // 128
        pad = torch.zeros(nb * 128, dtype=torch.float64, device=DEV)
        pad[:n] = x.abs()
        tpad = torch.zeros_like(pad)
        tpad[:n] = terms
        amax, tmax = pad.view(nb, 128).amax(1), tpad.view(nb, 128).amax(1)
        sf = s[name + "s"][i]
        within(sf, (amax / 448).clamp(min=1e-30), 8 * U * tmax / 448, f"{what} {name} scale")
        wide = sf.double().repeat_interleave(128)[:n]
        got = s[name][i].view(E4M3).double() * wide
        within(got, x, (2.0 ** -4 * x.abs() + 2.0 ** -10 * wide) * (1 + 2.0 ** -16) + 8 * U * terms, f"{what} {name}")


def clone(s):
    return {k: None if v is None else [t.clone() for t in v] for k, v in s.items()}


SIZES = [1, 2, 3, 4, 5, 127, 128, 129, 0, 1000, 2047, 2048, 2049, 6145, 100003]


@pytest.mark.parametrize("pt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("shift", [0, 1])
def test_step(pt, gt, q8, shift):
    s = tensors(SIZES, pt, gt, q8, copy=gt == torch.float32, seed=1, shift=shift)
    before = clone(s)
    refs = [step64(before["p"][i].double(), before["g"][i].double(), *states64(before, i), 7, 0.5, **HYPER)
            for i in range(len(SIZES))]
    gs = torch.full((1,), 0.5, device=DEV)
    bs.adamw_step(plan_of(s), step=7, grad_scale=gs, **HYPER)
    for i, n in enumerate(SIZES):
        if n:
            check_step(s, before, i, refs[i], f"tensor {i} ({n})")
        assert torch.equal(s["g"][i], before["g"][i])


@pytest.mark.parametrize("q8", [False, True])
def test_nothing_outside_the_tensors_is_written(q8):
    n, room = 1003, 64
    s = tensors([n], torch.float32, torch.float32, q8, True, 3)
    big = {}
    for k in ("p", "m", "v", "c"):
        b = torch.full((n + 2 * room,), 77, dtype=s[k][0].dtype, device=DEV)
        b[room:room + n] = s[k][0]
        big[k], s[k] = b, [b[room:room + n]]
    bs.adamw_step(plan_of(s), step=1, **HYPER)
    for k, b in big.items():
        assert bool((b[:room] == 77).all()) and bool((b[room + n:] == 77).all()), k


def test_zero_states_and_zero_gradients_start():
    """The first step from zeroed 8-bit states, and a block whose gradients are all zero."""
    s = tensors([384], torch.float32, torch.float32, True, False, 4)
    for k in ("m", "v", "ms", "vs"):
        s[k][0].zero_()
    s["g"][0][128:256] = 0
    before = clone(s)
    ref = step64(before["p"][0].double(), before["g"][0].double(), *states64(before, 0), 1, **HYPER)
    bs.adamw_step(plan_of(s), step=1, **HYPER)
    check_step(s, before, 0, ref)
    assert not s["m"][0][128:256].any() and not s["v"][0][128:256].any()


def test_factors_per_tensor():
    s = tensors([300, 300], torch.float32, torch.float32, False, False, 5)
    before = clone(s)
    bs.adamw_step(plan_of(s, lr_scales=[1.0, 0.5], decay_scales=[0.0, 1.0]), step=3, **HYPER)
    for i, h in enumerate((dict(HYPER, weight_decay=0.0), dict(HYPER, lr=HYPER["lr"] * 0.5))):
        check_step(s, before, i, step64(before["p"][i].double(), before["g"][i].double(), *states64(before, i), 3, **h))


def test_noop_flag():
    s = tensors([1000, 5], torch.float32, torch.bfloat16, True, True, 6)
    s["g"][0][3] = float("nan")
    before = clone(s)
    flag = torch.ones(1, device=DEV)
    plan = plan_of(s)
    bs.adamw_step(plan, step=2, noop_flag=flag, **HYPER)
    for k in s:
        for a, b in zip(s[k], before[k]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), k


@pytest.mark.parametrize("q8", [False, True])
def test_graph_with_device_step_and_rate(q8):
    """A captured step replayed with new gradients, step and rate equals the eager step bit for bit."""
    sizes = [5, 4100, 128]
    s = tensors(sizes, torch.float32, torch.float32, q8, True, 7)
    e = clone(s)
    plan, eager = plan_of(s), plan_of(e)
    lr, step = torch.zeros(1, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    h = {k: v for k, v in HYPER.items() if k != "lr"}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bs.adamw_step(plan, 0.0, step_dev=step, lr_dev=lr, **h)
    for t in range(1, 5):
        rate = torch.tensor(1e-3 * t, dtype=torch.float32)
        lr.fill_(float(rate))
        step.fill_(t)
        for a, b in zip(s["g"], e["g"]):
            a.copy_(torch.randn_like(a))
            b.copy_(a)
        graph.replay()
        torch.cuda.synchronize()
        bs.adamw_step(eager, float(rate), step=t, **h)
        for k in s:
            if s[k] is not None:
                for a, b in zip(s[k], e[k]):
                    assert torch.equal(a, b), (t, k)


def test_many_tensors_and_other_stream():
    sizes = [(i * 37) % 900 + 1 for i in range(1500)]
    s = tensors(sizes, torch.float32, torch.float32, False, False, 8)
    before = clone(s)
    side = torch.cuda.Stream()
    plan = plan_of(s)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        bs.adamw_step(plan, step=2, **HYPER)
    side.synchronize()
    flat = {k: [torch.cat(before[k]).double()] for k in ("p", "g", "m", "v")}
    ref = step64(flat["p"][0], flat["g"][0], flat["m"][0], flat["v"][0], 2, **HYPER)
    new = {k: [torch.cat(s[k])] for k in ("p", "m", "v")}
    check_step(dict(new, ms=None, vs=None, c=None), {"p": [torch.cat(before["p"])]}, 0, ref)


def test_eight_bit_states_follow_fp32_states():
    """200 steps on a noisy quadratic: both kinds of state reach the same loss (within a factor of 2)."""
    n = 4096
    g = torch.Generator(device=DEV).manual_seed(2)
    target, width = torch.randn(n, generator=g, device=DEV), torch.rand(n, generator=g, device=DEV) + 0.1
    loss = []
    for q8 in (False, True):
        s = tensors([n], torch.float32, torch.float32, q8, False, 9)
        for k in ("p", "m", "v", "ms", "vs"):
            if s[k] is not None:
                s[k][0].zero_()
        plan = plan_of(s)
        for t in range(1, 201):
            s["g"][0].copy_(width * (s["p"][0] - target) + 0.1 * torch.randn(n, generator=g, device=DEV))
            bs.adamw_step(plan, 2e-2, 0.9, 0.95, 1e-8, 0.0, t)
        loss.append(float((width * (s["p"][0] - target).square()).mean()))
    assert loss[1] < 2 * loss[0] and loss[0] < 0.05
