"""The gated projection at sizes that take each of its tiles: 256 x 256, and 128 x 128 with either K step at few and at many
tiles, in the forward; 128 x 128 at many tiles in the gradient.

Operands, checks and tolerances are those of the other tests of the gated projection."""
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs
import test_gpu_glu_gemm as T
from gpu_util import DEV, flush

pytestmark = pytest.mark.gpu

CASES = [(64, 33000, 96, 4128), (72, 32000, 416, 4256),  # 256 x 256 (the second: more groups than a wave's lanes)
         (20, 6000, 2080, 1056),                         # 128 x 128, many tiles, long K
         (9, 5000, 2080, 1056)]                          # 128 x 128, all tiles on the chip at once


@pytest.mark.parametrize("experts,rows,hidden,ffn", CASES)
def test_forward(experts, rows, hidden, ffn):
    flush(f"{experts} {rows} {hidden} {ffn}")
    s = T.operands(T.ragged(experts, rows, hidden), hidden, ffn, 41)
    R, n = s["R"], s["T"]
    ab = torch.full((R, 2 * ffn), float("nan"), dtype=torch.bfloat16, device=DEV)
    y = torch.full((R, ffn), float("nan"), device=DEV)
    out = T.poisoned(R, ffn, experts)
    bs.grouped_gemm_swiglu(s["xq"], hidden, s["w1q"], ffn, s["st"], R, probs=s["p"], ab=ab, y=y, y_dtype=bs.OUT_F32, out=out)
    rab, tab, ry, ty = T.forward64(s)
    T.within(ab[:n], rab, 2.0 ** -8 * rab.abs() + 1.01 * tab, "ab")
    T.within(y[:n], ry, ty, "y")
    assert bool(ab[n:].isnan().all()) and bool(y[n:].isnan().all())
    T.check_exact_quantization(out, y, s)
    T.check_untouched(out, s, ffn)


@pytest.mark.parametrize("experts,rows,hidden,ffn", CASES)
def test_gradient(experts, rows, hidden, ffn):
    flush(f"{experts} {rows} {hidden} {ffn}")
    s = T.operands(T.ragged(experts, rows, hidden + 1), hidden, ffn, 43)
    R, n = s["R"], s["T"]
    dab = torch.full((R, 2 * ffn), float("nan"), dtype=torch.bfloat16, device=DEV)
    dp = torch.full((R,), float("nan"), device=DEV)
    out = T.poisoned(R, 2 * ffn, experts)
    bs.grouped_gemm_swiglu_grad(s["xq"], hidden, s["w2q"], ffn, s["ab"], s["st"], R, probs=s["p"], dab=dab, out=out, dprobs=dp)
    rd, td, rp, tp = T.backward64(s)
    T.within(dab[:n], rd, 2.0 ** -8 * rd.abs() + 1.01 * td, "dab")
    T.within(dp[:n], rp, tp, "dprobs")
    assert bool(dab[n:].isnan().all()) and bool(dp[n:].isnan().all())
    T.check_close_quantization(out, rd, td, s)
    T.check_untouched(out, s, 2 * ffn)
