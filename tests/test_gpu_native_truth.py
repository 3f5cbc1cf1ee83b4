"""An `accumulate` whose truth is an error raises that error, as on the ctypes path."""
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("native", [True, False])
def test_truth_of_accumulate(monkeypatch, native):
    if not native:
        monkeypatch.setattr(bs, "_native", None)
    x = torch.randn((3, 16), device="cuda").bfloat16()
    f = bs.residual_norm(x, pre_weight=torch.ones(16, device="cuda"))
    with pytest.raises(RuntimeError, match="ambiguous"):
        bs.residual_norm_grad(x, None, f["r"], f["rstd_r"], torch.ones(16, device="cuda"), dpre_weight=torch.zeros(16, device="cuda"),
                              accumulate=torch.ones(2))
