"""The gradient of the residual norms written over its inputs: the same bits as into new tensors, also where dx overflows.

Row lengths that are not a multiple of 8: a row's last thread then holds elements of its neighbour's, which may be in another
wave (513 to 519 columns, the last thread being the first of its wave) or in its own."""
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("cols", [9, 15, 63, 511, 513, 516, 519, 1027, 2050, 4097, 8191])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("with_n", [False, True])
def test_gradient_in_place(cols, stream, with_n):
    rows = 300
    g = torch.Generator(device=DEV).manual_seed(cols)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    x, y, dn, dr = (rand(rows, cols).to(t) for t in (stream, torch.bfloat16, torch.bfloat16, stream))
    post, pre, gate = rand(cols), rand(cols), rand(cols)
    dr[::3] *= 2.0 ** 120  # x_scale takes these rows' dx to infinity
    kw = dict(y=y, post_weight=post, gate=gate, gate_kind=bs.GATE_CHANNEL, x_scale=2.0 ** 20, y_scale=2.0 ** -100)
    f = bs.residual_norm(x, y, post, pre, gate, bs.GATE_CHANNEL)
    kw["rstd_y"] = f["rstd_y"]
    if with_n:
        kw.update(r=f["r"], rstd_r=f["rstd_r"], pre_weight=pre)
    want = bs.residual_norm_grad(dn if with_n else None, dr, **kw)
    assert bool(want["dx"][::3].isinf().any()) and bool(want["dy"].isfinite().all())
    dx, dy = dr.clone(), dn.clone()
    got = bs.residual_norm_grad(dy if with_n else None, dx, dx=dx, dy=dy, **kw)
    assert got["dx"] is dx and got["dy"] is dy
    for k in want:
        assert torch.equal(got[k], want[k]), k
