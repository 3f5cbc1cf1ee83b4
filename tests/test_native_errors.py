"""A launch that failed on the native path is reported and not made again on the other one (no GPU needed: both paths
are replaced)."""
import types

import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

LAUNCH = -8


@pytest.fixture
def ctypes_calls(monkeypatch):
    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or 0

    library = bs.lib()
    failed = types.SimpleNamespace(**{n: lambda *a: LAUNCH for n in ("residual_norm", "residual_norm_grad", "swiglu",
                                                                     "swiglu_grad")})
    monkeypatch.setattr(bs, "_native", failed)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(bs, "_stream", lambda s: 0)
    monkeypatch.setattr(bs, "lib", Lib)
    monkeypatch.setattr(bs, "strerror", lambda code: library.bsfp8_strerror(code).decode())
    monkeypatch.setattr(bs, "_dev", lambda t, *a: 1 << 20)
    monkeypatch.setattr(bs, "_buf", lambda *a: 1 << 20)
    return calls


def test_reported_once(ctypes_calls):
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64)
    rows, splits = torch.zeros(4), torch.tensor([4], dtype=torch.int32)
    for call in (lambda: bs.residual_norm(x, pre_weight=w, r=x),
                 lambda: bs.residual_norm_grad(x, x, x, rows, w, dx=x, dpre_weight=w, accumulate=True),
                 lambda: bs.grouped_gemm_swiglu({}, 64, {}, 64, splits, 4, y=x),
                 lambda: bs.grouped_gemm_swiglu_grad({}, 64, {}, 64, x, splits, 4, dab=x)):
        with pytest.raises(bs.BSFP8Error, match="launch"):
            call()
        assert not ctypes_calls
