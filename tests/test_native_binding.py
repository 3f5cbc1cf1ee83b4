"""The native host path answers None for what it does not take, before any HIP call (no GPU needed)."""
import torch

import block_scaled_fp8_grouped_amd as bs


def test_built_and_hands_back():
    assert bs._native is not None, "build with __graft_entry__.build()"
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64)
    none = [None] * 4
    assert bs._native.residual_norm(x, None, None, w, None, 0, 1.0, 1.0, 1e-6, 0.0, *none, 0) is None
    assert bs._native.residual_norm("x", None, None, w, None, 0, 1.0, 1.0, 1e-6, 0.0, *none, 0) is None
    assert bs._native.residual_norm(x) is None and bs._native.residual_norm() is None
    assert bs._native.residual_norm_grad() is None and bs._native.residual_norm_grad(*[None] * 21) is None
    assert bs._native.swiglu() is None and bs._native.swiglu(*[None] * 19) is None
    assert bs._native.swiglu_grad() is None and bs._native.swiglu_grad(*[None] * 20) is None
    q = {"row_q": torch.zeros((4, 64), dtype=torch.uint8), "row_s": torch.zeros((2, 4), dtype=torch.uint8)}
    splits = torch.tensor([4], dtype=torch.int32)
    args = [q["row_q"], q["row_s"], 4, 64, q["row_q"], q["row_s"], 64, splits, bs.RECIPE_MX, bs.OUT_BF16] + [None] * 8
    assert bs._native.swiglu(*args, 0) is None
    for bad in (-1, 1 << 50, "4", None, 2.5):
        assert bs._native.swiglu(*(args[:2] + [bad] + args[3:]), 0) is None
