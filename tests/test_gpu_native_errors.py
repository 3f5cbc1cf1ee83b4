"""An error that the HIP runtime holds when a call launches (here that of an API call refused on the host) is reported by
that call, which is not made a second time: its in-place outputs and accumulated sums would not be its inputs any more."""
import ctypes

import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("native", [True, False])
def test_pending_error_is_reported(monkeypatch, native):
    if not native:
        monkeypatch.setattr(bs, "_native", None)
    g = torch.Generator(device=DEV).manual_seed(1)
    x, y = (torch.randn((40, 96), generator=g, device=DEV).bfloat16() for _ in range(2))
    w, ws = torch.randn(96, generator=g, device=DEV), torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    splits = torch.tensor([40], dtype=torch.int32, device=DEV)
    xq = bs.grouped_quantize(x, splits, bs.RECIPE_MX, bs.ROWWISE, bs.alloc_quantized(40, 96, 1, bs.RECIPE_MX, bs.ROWWISE))
    wq = bs.grouped_quantize(torch.randn((128, 96), generator=g, device=DEV).bfloat16(), None, bs.RECIPE_MX, bs.ROWWISE,
                             bs.alloc_quantized(128, 96, 1, bs.RECIPE_MX, bs.ROWWISE))
    f = bs.residual_norm(x, y, w, w)
    out = {k: torch.empty_like(v) for k, v in f.items()}
    glu = torch.empty((40, 64), dtype=torch.bfloat16, device=DEV)
    dr, sums = y.clone(), {k: torch.zeros(96, device=DEV) for k in ("dpre_weight", "dpost_weight")}
    grad = (x, dr, f["r"], f["rstd_r"], w, y, f["rstd_y"], w)
    dy = torch.empty_like(y)
    hip_set_device = bs.lib().hipSetDevice  # of the runtime that the library is linked with
    hip_set_device.argtypes, hip_set_device.restype = [ctypes.c_int], ctypes.c_int
    for call in (lambda: bs.residual_norm(x, y, w, w, **out),
                 lambda: bs.residual_norm_grad(*grad, dx=dr, dy=dy, accumulate=True, workspace=ws, **sums),
                 lambda: bs.grouped_gemm_swiglu(xq, 96, wq, 64, splits, 40, y=glu)):
        call()
        torch.cuda.synchronize()
        assert hip_set_device(1 << 20) != 0  # no such device: refused, the current one stays
        with pytest.raises(bs.BSFP8Error, match="launch"):
            call()
        torch.cuda.synchronize()
        call()
    torch.cuda.synchronize()
