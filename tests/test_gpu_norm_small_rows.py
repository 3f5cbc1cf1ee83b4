"""Norms without eps (or with one far below the rows) of rows whose mean square is a subnormal fp32 number.

Tolerance.  Every rounding of a subnormal sum is off by up to 2^-150; a mean of `cols` squares by twice that (the sums,
and the division), so rstd by 2^-150 / mean square of its value, beside the 2^-17 of the statistics of ordinary rows; an
output has that and half a step of its type."""
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("size", [1e-15, 1e-18, 2e-19, 1e-19, 3e-20, 1e-20])
@pytest.mark.parametrize("cols", [7, 40, 513, 2050, 9000, 16400])
@pytest.mark.parametrize("eps", [0.0, 1e-43])
def test_forward_and_gradient(size, cols, eps):
    g = torch.Generator(device=DEV).manual_seed(cols)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    x, w = rand(5, cols) * size, rand(cols)
    y = (rand(5, cols) * size).bfloat16()
    f = bs.residual_norm(x, y, pre_weight=w, post_weight=w, y_scale=size, eps=eps)
    ms = [t.double().square().mean(1) for t in (y, x.double() + size * y.double() / (y.double().square().mean(1, True) + eps).sqrt() * w)]
    for name, m in zip(("rstd_y", "rstd_r"), ms):
        want = (m + eps).rsqrt()
        off = (f[name].double() / want - 1).abs()
        # (rstd_r's r is itself off by rstd_y's share)
        tol = 2.0 ** -16 + 2.0 ** -149 / ms[0].min() + 2.0 ** -149 / m
        assert bool((off <= tol).all()), (name, float((off / tol).max()))
    r = f["r"].double()
    n = r * f["rstd_r"].double()[:, None] * w.double()
    assert bool(((f["n"].double() - n).abs() <= 2.0 ** -8 * n.abs() + 2.0 ** -17 * n.abs() + 1e-30).all())
    b = bs.residual_norm_grad(f["n"], None, f["r"], f["rstd_r"], w)
    assert bool(b["dx"].isfinite().all()) and bool(b["dpre_weight"].isfinite().all())


def test_rows_of_zeros_without_eps_are_not_numbers():
    """0 / 0, as the formula has it; the other rows of the call are not touched by it."""
    x, w = torch.zeros((3, 64), device=DEV), torch.ones(64, device=DEV)
    x[1] = 1
    f = bs.residual_norm(x, pre_weight=w, eps=0.0)
    assert bool(f["n"][0].isnan().all()) and bool((f["n"][1] == 1).all()) and bool(f["n"][2].isnan().all())
