"""Arrays of more than 2^31 elements: the last rows come out as those of a call on them alone, bit for bit."""
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


def test_norms():
    cols, tail = 8192, 40
    rows = (1 << 31) // cols + 77
    s = {k: torch.zeros((rows, cols), dtype=BF16, device=DEV) for k in ("x", "y", "dn", "dr")}
    for k in s:
        s[k][-tail:] = torch.randn((tail, cols), device=DEV).to(BF16)
    w = {k: torch.randn(cols, device=DEV) for k in ("post_weight", "pre_weight", "gate")}
    kw = dict(w, gate_kind=bs.GATE_CHANNEL)

    def both(part):
        f = bs.residual_norm(part["x"], part["y"], **kw)
        b = bs.residual_norm_grad(part["dn"], part["dr"], f["r"], f["rstd_r"], y=part["y"], rstd_y=f["rstd_y"], **kw)
        return {k: v[-tail:].clone() for k, v in dict(f, dx=b["dx"], dy=b["dy"]).items()}

    big, small = both(s), both({k: v[-tail:].clone() for k, v in s.items()})
    for k in small:
        assert torch.equal(big[k], small[k]), k
    assert bool(small["dx"].any())


def test_adamw():
    n, tail = (1 << 31) + 5000, 4096  # the tail begins at a block of 128
    first = (n - tail) // 128 * 128

    def state(count):
        return dict(p=torch.zeros(count, dtype=BF16, device=DEV), g=torch.zeros(count, dtype=BF16, device=DEV),
                    m=torch.zeros(count, dtype=torch.uint8, device=DEV), v=torch.zeros(count, dtype=torch.uint8, device=DEV),
                    ms=torch.zeros((count + 127) // 128, device=DEV), vs=torch.zeros((count + 127) // 128, device=DEV))

    big, small = state(n), state(n - first)
    for k in ("p", "g"):
        small[k].copy_(torch.randn(n - first, device=DEV))
        big[k][first:] = small[k]
    for s in (big, small):
        plan = bs.adamw_plan([s["p"]], [s["g"]], [s["m"]], [s["v"]], [s["ms"]], [s["vs"]])
        bs.adamw_step(plan, 1e-2, step=1)
    for k in ("p", "m", "v"):
        assert torch.equal(big[k][first:], small[k]), k
    for k in ("ms", "vs"):
        assert torch.equal(big[k][first // 128:], small[k]), k
    assert not bool(big["p"][:first].any())


def test_gated_projection():
    """ab and (da | db) of more than 2^31 elements; the groups are one large and one of the last 300 rows."""
    hidden, ffn, tail = 32, 16384, 300
    rows = (1 << 31) // (2 * ffn) + 500
    g = torch.Generator(device=DEV).manual_seed(2)
    codes = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8, device=DEV) & 0xB7  # noqa: E731 (small finite)
    both = bs.ROWWISE | bs.COLWISE

    def scale(*s):
        return torch.full(s, 127, dtype=torch.uint8, device=DEV)

    x = {"row_q": codes(rows, hidden), "row_s": scale(1, rows)}
    w1 = codes(2 * ffn, hidden)
    w2, w2s = codes(ffn * 128).view(ffn, 128), scale(4, ffn)
    w2[:, hidden:] = 0

    def call(part, splits):
        E, R = len(splits), part["row_q"].shape[0]
        st = torch.tensor(splits, dtype=torch.int32, device=DEV)
        wq = {"row_q": w1.repeat(E, 1), "row_s": scale(1, E * 2 * ffn)}
        wc = {"col_q": w2.reshape(-1).repeat(E), "col_s": w2s.reshape(-1).repeat(E)}
        ab = torch.zeros((R, 2 * ffn), dtype=BF16, device=DEV)
        q = bs.alloc_quantized(R, ffn, E, bs.RECIPE_MX, both)
        bs.grouped_gemm_swiglu(part, hidden, wq, ffn, st, R, ab=ab, out=q)
        dab, dp = torch.zeros_like(ab), torch.zeros(R, device=DEV)
        dq = bs.alloc_quantized(R, 2 * ffn, E, bs.RECIPE_MX, both)
        bs.grouped_gemm_swiglu_grad(part, hidden, wc, ffn, ab, st, R, dab=dab, out=dq, dprobs=dp)
        kp = (tail + 127) // 128 * 128
        at = sum((k + 127) // 128 * 128 for k in splits[:-1])
        r = {"ab": ab[-tail:], "dab": dab[-tail:], "dprobs": dp[-tail:]}
        for name, o, c in (("q", q, ffn), ("dq", dq, 2 * ffn)):
            r.update({name + "_row": o["row_q"][-tail:], name + "_rows": o["row_s"][:, -tail:],
                      name + "_col": o["col_q"][c * at:c * (at + kp)], name + "_cols": o["col_s"][c * at // 32:c * (at + kp) // 32]})
        return {k: v.clone() for k, v in r.items()}

    big = call(x, [rows - tail, tail])
    small = call({"row_q": x["row_q"][-tail:].clone(), "row_s": scale(1, tail)}, [tail])
    for k in small:
        # (other tiles, whose sums over a single scale block of 32 terms run in the same order; dprobs' columns are
        # added in another)
        if k == "dprobs":
            assert torch.allclose(big[k], small[k], rtol=1e-4, atol=1e-3 * float(small[k].abs().max()))
        else:
            assert torch.equal(big[k], small[k]), k
    assert bool(small["dab"].any())
