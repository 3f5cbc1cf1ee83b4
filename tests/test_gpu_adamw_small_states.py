"""8-bit states of elements far below their block's largest: sqrt(v) keeps a nonzero code where it is not zero, since m, whose
scale is its own, may, and the next step divides by it."""
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def fresh(n, q8):
    z = lambda c=n, t=torch.float32: torch.zeros(c, dtype=t, device=DEV)  # noqa: E731
    s = dict(p=z(), g=z())
    if q8:
        s.update(m=z(t=torch.uint8), v=z(t=torch.uint8), ms=z(n // 128), vs=z(n // 128))
        return s, bs.adamw_plan([s["p"]], [s["g"]], [s["m"]], [s["v"]], [s["ms"]], [s["vs"]])
    s.update(m=z(), v=z())
    return s, bs.adamw_plan([s["p"]], [s["g"]], [s["m"]], [s["v"]])


@pytest.mark.parametrize("seed", [None, 5])
def test_nonzero_states_keep_nonzero_codes(seed):
    n = 4096
    s, plan = fresh(n, True)
    s["g"].copy_(10.0 ** (-9 * torch.rand(n, device=DEV)))  # sqrt(v) from far below the smallest code up
    s["g"].view(-1, 128)[:, 0] = 1
    s["g"].view(-1, 128)[:, 1:9] = 0
    for t in range(1, 4):
        bs.adamw_step(plan, 1e-3, beta2=0.999, step=t, seed=seed)
        zero = s["g"] == 0
        assert not bool(s["v"][zero].any()) and bool((s["v"][~zero] > 0).all())
        assert bool((s["v"][~zero] < 0x7f).all())


def test_updates_stay_within_those_of_fp32_states():
    """Gradients of 1e-6 beside one that alternates between 1 and -1, and a last step without them.  sqrt(v) is never
    stored below its value here, and m (4 of the lowest codes) no further off than half a code: 1 / 8 of it."""
    (a, plan), (b, plain) = fresh(128, True), fresh(128, False)
    lr = 1e-3
    for t in range(1, 301):
        for s in (a, b):
            s["g"].fill_(1e-6 if t < 300 else 0.0)
            s["g"][0] = 1.0 if t % 2 else -1.0
            s["p"].zero_()
        bs.adamw_step(plan, lr, beta2=0.999, step=t, weight_decay=0.0)
        bs.adamw_step(plain, lr, beta2=0.999, step=t, weight_decay=0.0)
        assert bool((a["p"][1:].abs() <= 1.125 * b["p"][1:].abs()).all()), (t, float(a["p"][1] / lr), float(b["p"][1] / lr))
