"""Few rows in more groups than a wave has lanes: the few-rows kernel places its tiles by the workgroup's scan there.

Operands and tolerances are those of the other tests of the gated projection."""
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs
import test_gpu_glu_gemm as T
from gpu_util import DEV, flush

pytestmark = pytest.mark.gpu


def sizes(experts, rows):
    """`rows` rows over every third expert and, unequally, the first and the last one."""
    k = [0] * experts
    for i in range(rows):
        k[(3 * i) % experts if i % 4 else (0 if i % 8 else experts - 1)] += 1
    return k


CASES = [(65, 9), (65, 300), (100, 1), (128, 128), (128, 1000), (257, 40), (1024, 700)]


@pytest.mark.parametrize("experts,rows", CASES)
@pytest.mark.parametrize("hidden,ffn", [(32, 32), (160, 96)])
def test_forward(experts, rows, hidden, ffn):
    flush(f"{experts} {rows} {hidden} {ffn}")
    s = T.operands(sizes(experts, rows), hidden, ffn, experts + rows)
    R = s["R"]
    assert R <= 12 * experts  # the tile rule's few rows
    ab = torch.full((R, 2 * ffn), float("nan"), dtype=torch.bfloat16, device=DEV)
    y = torch.full((R, ffn), float("nan"), device=DEV)
    out = T.poisoned(R, ffn, experts)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    bs.grouped_gemm_swiglu(s["xq"], hidden, s["w1q"], ffn, s["st"], R, probs=s["p"], ab=ab, y=y, y_dtype=bs.OUT_F32, out=out,
                           status=status)
    assert int(status.item()) == 0
    rab, tab, ry, ty = T.forward64(s)
    n = s["T"]
    T.within(ab[:n], rab, 2.0 ** -8 * rab.abs() + 1.01 * tab, "ab")
    T.within(y[:n], ry, ty, "y")
    assert bool(ab[n:].isnan().all()) and bool(y[n:].isnan().all())
    T.check_exact_quantization(out, y, s)
    T.check_untouched(out, s, ffn)


@pytest.mark.parametrize("experts,rows", CASES)
@pytest.mark.parametrize("hidden,ffn", [(32, 32), (160, 96)])
def test_gradient(experts, rows, hidden, ffn):
    flush(f"{experts} {rows} {hidden} {ffn}")
    s = T.operands(sizes(experts, rows), hidden, ffn, experts + rows + 1)
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


def test_bad_sizes_write_nothing():
    s = T.operands(sizes(100, 50), 96, 64, 11)
    for change, bit in ((-1, bs.STATUS_NEGATIVE_SPLIT), (1 << 30, bs.STATUS_EXCEEDS_CAPACITY)):
        st = s["st"].clone()
        st[70] = change
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        y, dp = torch.full((s["R"], 64), 7.0, device=DEV), torch.full((s["R"],), 7.0, device=DEV)
        bs.grouped_gemm_swiglu(s["xq"], 96, s["w1q"], 64, st, s["R"], y=y, y_dtype=bs.OUT_F32, status=status)
        assert int(status.item()) == bit and bool((y == 7).all())
        status.zero_()
        bs.grouped_gemm_swiglu_grad(s["xq"], 96, s["w2q"], 64, s["ab"], st, s["R"], dprobs=dp, status=status)
        assert int(status.item()) == bit and bool((dp == 7).all())
