"""The default stream given by its handle, 0, or as an object: the calls that make a given stream the current one run
there, and elsewhere than the stream that is current meanwhile."""
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def glu_operands(tokens=9, hidden=96, ffn=1056, experts=3):
    g = torch.Generator(device=DEV).manual_seed(6)
    u8 = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8, device=DEV) & 0xB7  # noqa: E731
    one = lambda *s: torch.full(s, 120, dtype=torch.uint8, device=DEV)  # noqa: E731
    splits = torch.tensor([4, 0, 5], dtype=torch.int32, device=DEV)
    ab = torch.randn((tokens, 2 * ffn), generator=g, device=DEV).bfloat16()
    return ({"row_q": u8(tokens, hidden), "row_s": one(hidden // 32, tokens)}, hidden,
            {"col_q": u8(experts * ffn * 128), "col_s": one(experts * ffn * 4)}, ffn, ab, splits, tokens)


@pytest.mark.parametrize("given", [0, "object", "handle"])
@pytest.mark.parametrize("native", [True, False])
def test_default_stream(monkeypatch, given, native):
    default = torch.cuda.default_stream()
    stream = {0: 0, "object": default, "handle": default.cuda_stream}[given]
    if not native:
        monkeypatch.setattr(bs, "_native", None)
    g = torch.Generator(device=DEV).manual_seed(5)
    x, y = (torch.randn((300, 520), generator=g, device=DEV).bfloat16() for _ in range(2))
    w = torch.randn(520, generator=g, device=DEV)
    glu = glu_operands()
    R, F = glu[-1], glu[3]
    assert bs.grouped_gemm_swiglu_grad_workspace_bytes(R, F, 3) > 0
    seen = []
    raw = bs._stream
    monkeypatch.setattr(bs, "_stream", lambda s: seen.append(raw(s)) or seen[-1])

    dprobs = [torch.zeros(R, device=DEV) for _ in range(2)]

    def calls(dp, **kw):
        f = bs.residual_norm(x, y, w, w, **kw)
        b = bs.residual_norm_grad(y, x, f["r"], f["rstd_r"], w, y, f["rstd_y"], w, **kw)
        p = bs.grouped_gemm_swiglu_grad(*glu, dprobs=dp, **kw)
        return {**f, **b, **p}

    want = calls(dprobs[0])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # (nothing runs on it: all tensors belong to the default stream)
        seen.clear()
        launched = calls(dprobs[1], stream=stream)
        # the last handle that each of the three calls looked up is the one that it launched on
        assert seen[-1] == 0 and seen.count(0) >= 3
    torch.cuda.synchronize()
    for k, t in launched.items():
        assert torch.equal(t, want[k]), k
