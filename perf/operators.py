"""The operators of one training step around the grouped GEMMs of an expert layer, as cases that can be
timed and compared: the gated feed-forward projection and its gradient, the norms around a block with its
gate and residual scale and their gradient, and the AdamW step over many tensors.

`run` computes a case in plain torch operations, or, where `own` is true, with this framework's kernels.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3, E8M0, BF16, F32, F64 = torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.bfloat16, torch.float32, torch.float64
GLU = ("glu", "glu_grad")


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------

def listed():
    return [
        # serving one token: 8 of 32 experts get one row each; bounded by reading their weights
        {"name": "swiglu_token", "op": "glu", "experts": 32, "empty": 24, "tokens": 8, "pad": 0, "hidden": 7168,
         "ffn": 2048, "out": "bf16"},
        # a small training step on few experts, one of them empty, padded buffer, hidden not a multiple of 128
        {"name": "swiglu_step", "op": "glu", "experts": 8, "empty": 1, "tokens": 4099, "pad": 61, "hidden": 4128,
         "ffn": 1024, "out": "mxfp8"},
        # a training step's expert layer on one GPU of an expert-parallel group
        {"name": "swiglu_layer", "op": "glu", "experts": 32, "empty": 2, "tokens": 65536, "pad": 0, "hidden": 4096,
         "ffn": 2048, "out": "mxfp8"},
        # the gradients of the last two, from the gradient that arrives at the second projection's output
        {"name": "swiglu_grad_step", "op": "glu_grad", "experts": 8, "empty": 1, "tokens": 4099, "pad": 61,
         "hidden": 4128, "ffn": 1024, "out": "bf16"},
        {"name": "swiglu_grad_layer", "op": "glu_grad", "experts": 32, "empty": 2, "tokens": 65536, "pad": 0,
         "hidden": 4096, "ffn": 2048, "out": "mxfp8"},
        # norms around a block while serving four tokens: latency
        {"name": "norm_tokens", "op": "norm", "rows": 4, "cols": 7168, "stream": "bf16", "gate": "channel"},
        # the same in training, bf16 and fp32 residual streams, and its gradient
        {"name": "norm_layer", "op": "norm", "rows": 32768, "cols": 7168, "stream": "bf16", "gate": "channel"},
        {"name": "norm_grad_odd", "op": "norm_grad", "rows": 4099, "cols": 2050, "stream": "fp32", "gate": "token"},
        {"name": "norm_grad_layer", "op": "norm_grad", "rows": 32768, "cols": 7168, "stream": "bf16",
         "gate": "channel"},
        # the small tensors of a model (norm weights, gates, routers' rows): one launch for all
        {"name": "adamw_small", "op": "adamw", "state": "fp32", "param": "fp32", "grad": "fp32", "copy": False,
         "tensors": 301, "low": 1, "high": 8192, "mix": 1},
        # expert weights: fp32 master weights and main_grad, a bf16 copy for the next quantize
        {"name": "adamw_layer", "op": "adamw", "state": "fp32", "param": "fp32", "grad": "fp32", "copy": True,
         "tensors": 12, "low": 1 << 23, "high": 1 << 26, "mix": 2},
        # the same weights with 8-bit states
        {"name": "adamw_layer_8bit", "op": "adamw", "state": "8bit", "param": "fp32", "grad": "fp32", "copy": True,
         "tensors": 12, "low": 1 << 23, "high": 1 << 26, "mix": 2},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["glu", "glu_grad", "norm", "norm_grad", "adamw"])
    if op in GLU:
        experts = log(1, 64)
        c = {"op": op, "experts": experts, "empty": rng.randint(0, experts // 2), "tokens": log(1, 32768),
             "pad": rng.choice([0, rng.randint(1, 300)]), "hidden": 32 * log(8, 224), "ffn": 32 * log(4, 64),
             "out": rng.choice(["bf16", "mxfp8"])}
        return c
    if op in ("norm", "norm_grad"):
        return {"op": op, "rows": log(1, 16384), "cols": log(33, 8192), "stream": rng.choice(["bf16", "fp32"]),
                "gate": rng.choice(["none", "channel", "token"])}
    low = log(1, 1 << 20)
    return {"op": op, "state": rng.choice(["fp32", "8bit"]), "param": rng.choice(["fp32", "bf16"]),
            "grad": rng.choice(["fp32", "bf16"]), "copy": rng.random() < 0.5, "tensors": log(1, 64), "low": low,
            "high": low * log(1, 8), "mix": rng.randint(0, 1 << 20)}


def _counts(case, seed):
    """Rows of each expert: the live experts get their tokens by a uniform draw (one each where there are
    as many tokens as live experts)."""
    rng = np.random.default_rng(seed)
    e, live, t = case["experts"], case["experts"] - case["empty"], case["tokens"]
    at = np.sort(rng.choice(e, live, replace=False))
    k = np.zeros(e, dtype=np.int64)
    k[at] = 1 if t == live else rng.multinomial(t, np.full(live, 1.0 / live))
    return k


def _sizes(case):
    r = random.Random(case["mix"])
    return [int(math.exp(r.uniform(math.log(case["low"]), math.log(case["high"] + 0.5))))
            for _ in range(case["tensors"])]


def _dtype(name):
    return {"fp32": F32, "bf16": BF16}[name]


def work(case):
    op = case["op"]
    if op in GLU:
        t, h, f = case["tokens"], case["hidden"], case["ffn"]
        live = min(t, case["experts"] - case["empty"])
        q = 33 / 32  # bytes of an MXFP8 value with its share of the scale
        if op == "glu":
            out = t * f * 2 if case["out"] == "bf16" else t * 2 * f * 2 + 2 * t * f * q
            return {"bytes": q * (t * h + live * 2 * f * h) + out + 4 * t, "flops": 4 * t * h * f}
        out = t * 2 * f * 2 if case["out"] == "bf16" else 2 * t * 2 * f * q
        return {"bytes": q * (t * h + live * f * h) + t * 2 * f * 2 + out + 8 * t, "flops": 2 * t * h * f}
    if op in ("norm", "norm_grad"):
        n, s = case["rows"] * case["cols"], 2 if case["stream"] == "bf16" else 4
        gate = 4 * (case["rows"] if case["gate"] == "token" else case["cols"] if case["gate"] == "channel" else 0)
        if op == "norm":
            return {"bytes": n * (2 * s + 4) + 8 * case["rows"] + 8 * case["cols"] + gate, "flops": 12 * n}
        return {"bytes": n * (3 * s + 6) + 8 * case["rows"] + 16 * case["cols"] + 2 * gate, "flops": 24 * n}
    n, p, g = sum(_sizes(case)), 2 if case["param"] == "bf16" else 4, 2 if case["grad"] == "bf16" else 4
    state = 16 if case["state"] == "fp32" else 4 * (1 + 4 / 128)
    return {"bytes": n * (2 * p + g + state + (2 if case["copy"] else 0)), "flops": 15 * n}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _mx_blocks(v):
    """MXFP8 of fp32 blocks of 32 along the last axis: e4m3 codes and E8M0 bytes."""
    b = v.unflatten(-1, (-1, 32))
    frac, e = torch.frexp(b.abs().amax(-1))
    e = torch.where(frac == 0, -127, (e - 9 + (frac > 0.875)).clamp(-127, 127))
    q = (b * torch.exp2(-e.to(F32)).unsqueeze(-1)).to(E4M3)
    return q.flatten(-2), (e + 127).to(torch.uint8)


def _randn(shape, g, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=F32) * scale


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    if op in GLU:
        e, t, h, f = case["experts"], case["tokens"], case["hidden"], case["ffn"]
        rows, counts = t + case["pad"], _counts(case, seed)
        s = {"op": op, "out": case["out"], "e": e, "t": t, "rows": rows, "h": h, "f": f, "most": int(counts.max()),
             "splits": torch.tensor(counts, dtype=torch.int32, device=DEV)}
        q, sc = _mx_blocks(_randn((t, h), g))
        # rows past the last expert's hold any bits
        s["x"] = {"row_q": torch.full((rows, h), 0x7f, dtype=torch.uint8, device=DEV),
                  "row_s": torch.full((h // 32, rows), 0xff, dtype=torch.uint8, device=DEV)}
        s["x"]["row_q"][:t] = q.view(torch.uint8)
        s["x"]["row_s"][:, :t] = sc.t()
        s["probs"] = torch.rand(rows, generator=g, device=DEV, dtype=F32)
        width = f if op == "glu" else 2 * f
        if op == "glu":
            q, sc = _mx_blocks(_randn((e * 2 * f, h), g, h ** -0.5))
            s["w"] = {"row_q": q.view(torch.uint8), "row_s": sc.t().contiguous()}
            if case["out"] == "mxfp8":
                s["ab"] = torch.zeros((rows, 2 * f), dtype=BF16, device=DEV)
        else:
            # the second projection [e, h, f], quantized along h: its codes per output channel f
            q, sc = _mx_blocks(_randn((e, f, h), g, f ** -0.5))
            wq = torch.zeros((e, f, (h + 127) // 128 * 128), dtype=torch.uint8, device=DEV)
            ws = torch.zeros((e, (h + 127) // 128 * 4, f), dtype=torch.uint8, device=DEV)
            wq[:, :, :h] = q.view(torch.uint8)
            ws[:, : h // 32] = sc.transpose(1, 2)
            s["w"] = {"col_q": wq.view(-1), "col_s": ws.view(-1)}
            s["ab"] = torch.zeros((rows, 2 * f), dtype=BF16, device=DEV)
            s["ab"][:t] = _randn((t, 2 * f), g).to(BF16)
            s["dprobs"] = torch.zeros(rows, dtype=F32, device=DEV)
        if case["out"] == "bf16":
            s["y"] = torch.zeros((rows, width), dtype=BF16, device=DEV)
        else:
            bound = 128 * ((rows + 127 * e) // 128)
            s["q"] = {"row_q": torch.zeros((rows, width), dtype=torch.uint8, device=DEV),
                      "row_s": torch.zeros((width // 32, rows), dtype=torch.uint8, device=DEV),
                      "col_q": torch.zeros(width * bound, dtype=torch.uint8, device=DEV),
                      "col_s": torch.zeros(width * bound // 32, dtype=torch.uint8, device=DEV)}
        return s
    if op in ("norm", "norm_grad"):
        r, c, st = case["rows"], case["cols"], _dtype(case["stream"])
        s = {"op": op, "gate_kind": case["gate"], "eps": 1e-6, "x_scale": 1.0, "y_scale": 0.5, "offset": 1.0}
        s["x"] = _randn((r, c), g, 3.0).to(st)
        s["y"] = _randn((r, c), g, 2.0).to(BF16)
        s["post"], s["pre"] = _randn((c,), g, 0.1), _randn((c,), g, 0.1)
        shape = {"none": None, "channel": (c,), "token": (r,)}[case["gate"]]
        s["gate"] = None if shape is None else torch.sigmoid(_randn(shape, g))
        if op == "norm_grad":
            s["r"] = s.pop("x")
            s["rstd_r"] = torch.rsqrt(s["r"].float().square().mean(1) + s["eps"])
            s["rstd_y"] = torch.rsqrt(s["y"].float().square().mean(1) + s["eps"])
            s["dn"] = _randn((r, c), g, 0.01).to(BF16)
            s["dr"] = _randn((r, c), g, 0.01).to(st)
        return s
    sizes = _sizes(case)
    at = np.cumsum([0] + [(n + 127) // 128 * 128 for n in sizes])
    total = int(at[-1])
    where = [(int(o), n) for o, n in zip(at, sizes)]
    # one arena each; a tensor begins at a multiple of 128 elements and the rest of its last 128 is zero
    live = torch.zeros(total, dtype=F32, device=DEV)
    live.copy_(torch.from_numpy(_live(where, total)))
    s = {"op": op, "state": case["state"], "lr": 2e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "decay": 0.1,
         "step": 11, "where": where}
    s["grad_scale"] = torch.full((1,), 0.7, dtype=F32, device=DEV)
    s["p"] = (_randn(total, g, 0.02) * live).to(_dtype(case["param"]))
    # gradients whose size differs from channel to channel, as weight gradients' do
    wide = torch.exp(_randn((total + 1023) // 1024, g, 2.0)).repeat_interleave(1024)[:total]
    s["g"] = (_randn(total, g, 1e-3) * wide * live).to(_dtype(case["grad"]))
    m, u = _randn(total, g, 3e-4) * wide * live, (_randn(total, g, 7e-4).abs() + 1e-4) * wide * live
    if case["state"] == "fp32":
        s["m"], s["v"] = m, u * u
    else:
        for name, x in (("m", m), ("v", u)):
            b = x.view(-1, 128)
            sf = (b.abs().amax(1) / 448).clamp(min=1e-30)
            s[name], s[name + "_s"] = (b / sf[:, None]).to(E4M3).view(-1).view(torch.uint8), sf
    if case["copy"]:
        s["copy"] = s["p"].to(BF16)
    if own:
        import block_scaled_fp8_grouped_amd as bs

        def parts(x):
            return [x[o:o + n] for o, n in where]

        def blocks(x):
            return [x[o // 128:(o + n + 127) // 128] for o, n in where]

        q = case["state"] == "8bit"
        s["plan"] = bs.adamw_plan(parts(s["p"]), parts(s["g"]), parts(s["m"]), parts(s["v"]),
                                  exp_avg_scales=blocks(s["m_s"]) if q else None,
                                  exp_avg_sq_scales=blocks(s["v_s"]) if q else None,
                                  copies=parts(s["copy"]) if case["copy"] else None)
    return s


def _live(where, total):
    v = np.zeros(total, dtype=np.float32)
    for o, n in where:
        v[o:o + n] = 1
    return v


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)(s)


def _outputs(s):
    """What a gated projection returns: 16-bit values as they are, MXFP8 as its values and its scales."""
    out = {}
    if "y" in s:
        out["y"] = s["y"]
    else:
        if s["op"] == "glu":
            out["ab"] = s["ab"]
        for k, v in s["q"].items():
            out[k] = v.view(E4M3 if k.endswith("_q") else E8M0)
    if s["op"] == "glu_grad":
        out["dprobs"] = s["dprobs"]
    return out


def _own(s):
    import block_scaled_fp8_grouped_amd as bs

    op = s["op"]
    if op == "glu":
        bs.grouped_gemm_swiglu(s["x"], s["h"], s["w"], s["f"], s["splits"], s["rows"], bs.RECIPE_MX, probs=s["probs"],
                               ab=s.get("ab"), y=s.get("y"), y_dtype=bs.OUT_BF16, out=s.get("q"))
        return _outputs(s)
    if op == "glu_grad":
        bs.grouped_gemm_swiglu_grad(s["x"], s["h"], s["w"], s["f"], s["ab"], s["splits"], s["rows"], bs.RECIPE_MX,
                                    probs=s["probs"], dab=s.get("y"), out=s.get("q"), dprobs=s["dprobs"])
        return _outputs(s)
    if op in ("norm", "norm_grad"):
        kind = {"none": bs.GATE_NONE, "channel": bs.GATE_CHANNEL, "token": bs.GATE_TOKEN}[s["gate_kind"]]
        more = dict(gate=s["gate"], gate_kind=kind, x_scale=s["x_scale"], y_scale=s["y_scale"],
                    weight_offset=s["offset"])
        if op == "norm":
            return bs.residual_norm(s["x"], s["y"], s["post"], s["pre"], eps=s["eps"], **more)
        return bs.residual_norm_grad(s["dn"], s["dr"], s["r"], s["rstd_r"], s["pre"], s["y"], s["rstd_y"], s["post"],
                                     **more)
    bs.adamw_step(s["plan"], s["lr"], s["beta1"], s["beta2"], s["eps"], s["decay"], s["step"],
                  grad_scale=s["grad_scale"])
    return _states(s)


def _states(s):
    out = {"p": s["p"]}
    if s["state"] == "fp32":
        out["m"], out["v"] = s["m"], s["v"]
    else:
        out["m"], out["v"], out["m_s"], out["v_s"] = s["m"].view(E4M3), s["v"].view(E4M3), s["m_s"], s["v_s"]
    if "copy" in s:
        out["copy"] = s["copy"]
    return out


def _values(q, scale):
    """fp32 values of e4m3 codes [..., n] and E8M0 bytes [..., n / 32]."""
    two = torch.exp2(scale.to(F32) - 127)
    return (q.view(E4M3).to(F32).unflatten(-1, (-1, 32)) * two.unsqueeze(-1)).flatten(-2)


def _places(s):
    """Each live row's expert, its place in the expert, and the expert's first row in the token buffer and in
    the layout whose experts begin at multiples of 128 rows."""
    k = s["splits"].long()
    kp = (k + 127) // 128 * 128
    of = torch.repeat_interleave(torch.arange(s["e"], device=DEV), k, output_size=s["t"])
    first, packed = k.cumsum(0) - k, kp.cumsum(0) - kp
    return of, torch.arange(s["t"], device=DEV) - first[of], packed[of], kp[of]


def _product(s, x, w, of, at):
    """x's rows times their own experts' w [e, n, k], in fp32: an expert's rows side by side, or where there
    are few rows each row's own weights."""
    t = s["t"]
    if t <= s["e"]:
        return torch.bmm(_values(w[0][of], w[1][of]), x.unsqueeze(2)).squeeze(2)
    rows = torch.zeros((s["e"], s["most"], s["h"]), dtype=F32, device=DEV)
    rows[of, at] = x
    return torch.bmm(rows, _values(*w).transpose(1, 2))[of, at]


def _keep(s, v, at, packed, kp):
    """An output [t, n] in fp32, kept in the forms that were asked for."""
    t, n = v.shape
    if "y" in s:
        s["y"][:t] = v.to(BF16)
        return
    q, sc = _mx_blocks(v)
    s["q"]["row_q"][:t] = q.view(torch.uint8)
    s["q"]["row_s"][:, :t] = sc.t()
    # blocks of 32 rows of one expert; the codes of a channel side by side
    bound = s["q"]["col_q"].numel() // n
    tall = torch.zeros((n, bound), dtype=F32, device=DEV)
    tall[:, packed + at] = v.t()
    q, sc = _mx_blocks(tall)
    s["q"]["col_s"].view(-1, n).copy_(sc.t())
    # (an expert's part of the buffer begins at n times its first row; within it a channel has kp codes)
    place = (n * packed + at).unsqueeze(1) + torch.arange(n, device=DEV) * kp.unsqueeze(1)
    s["q"]["col_q"][place] = q.view(torch.uint8)[:, packed + at].t()


def _plain(s):
    op = s["op"]
    if op in GLU:
        e, t, h, f = s["e"], s["t"], s["h"], s["f"]
        of, at, packed, kp = _places(s)
        x = _values(s["x"]["row_q"][:t], s["x"]["row_s"][:, :t].t())
        p = s["probs"][:t, None]
        if op == "glu":
            w = (s["w"]["row_q"].view(e, 2 * f, h), s["w"]["row_s"].t().reshape(e, 2 * f, h // 32))
            ab = _product(s, x, w, of, at)
            if "ab" in s:
                s["ab"][:t] = ab.to(BF16)
            a, b = ab[:, :f], ab[:, f:]
            _keep(s, a / (1 + torch.exp(-a)) * b * p, at, packed, kp)
            return _outputs(s)
        w = (s["w"]["col_q"].view(e, f, -1)[:, :, :h], s["w"]["col_s"].view(e, -1, f)[:, : h // 32].transpose(1, 2))
        dh = _product(s, x, w, of, at)
        a, b = s["ab"][:t, :f].float(), s["ab"][:t, f:].float()
        sg = 1 / (1 + torch.exp(-a))
        q = dh * p
        s["dprobs"][:t] = (dh * (a * sg) * b).sum(1)
        _keep(s, torch.cat([q * b * (sg * (1 + a * (1 - sg))), q * (a * sg)], 1), at, packed, kp)
        return _outputs(s)
    if op in ("norm", "norm_grad"):
        y, post, pre = s["y"].float(), s["post"] + s["offset"], s["pre"] + s["offset"]
        gate = s["gate"].view(-1, 1) if s["gate_kind"] == "token" else s["gate"] if s["gate_kind"] == "channel" else 1
        if op == "norm":
            x = s["x"].float()
            ry = torch.rsqrt(y.square().mean(1) + s["eps"])
            r = s["x_scale"] * x + s["y_scale"] * gate * (y * ry[:, None] * post)
            rr = torch.rsqrt(r.square().mean(1) + s["eps"])
            return {"r": r.to(s["x"].dtype), "n": (r * rr[:, None] * pre).to(BF16), "rstd_y": ry, "rstd_r": rr}
        dn, rr, ry = s["dn"].float(), s["rstd_r"][:, None], s["rstd_y"][:, None]
        rh, yh = s["r"].float() * rr, y * ry
        g1 = dn * pre
        d = s["dr"].float() + rr * (g1 - rh * (g1 * rh).mean(1, keepdim=True))
        back = s["y_scale"] * d
        dz = gate * back
        g2 = dz * post
        dy = ry * (g2 - yh * (g2 * yh).mean(1, keepdim=True))
        out = {"dx": (s["x_scale"] * d).to(s["r"].dtype), "dy": dy.to(BF16), "dpre_weight": (dn * rh).sum(0),
               "dpost_weight": (dz * yh).sum(0)}
        if s["gate_kind"] != "none":
            out["dgate"] = (back * yh * post).sum(1 if s["gate_kind"] == "token" else 0)
        return out
    return _plain_adamw(s)


def _plain_adamw(s):
    b1, b2 = s["beta1"], s["beta2"]
    g = s["g"].float() * s["grad_scale"]
    if s["state"] == "fp32":
        m, v = s["m"], s["v"]
    else:
        m = (s["m"].view(E4M3).float().view(-1, 128) * s["m_s"][:, None]).view(-1)
        v = (s["v"].view(E4M3).float().view(-1, 128) * s["v_s"][:, None]).view(-1).square()
    m = m * b1 + g * (1 - b1)
    v = v * b2 + g * g * (1 - b2)
    by = torch.sqrt(v) * ((1 - b2 ** s["step"]) ** -0.5) + s["eps"]
    p = s["p"].float() * (1 - s["lr"] * s["decay"]) - m / by * (s["lr"] / (1 - b1 ** s["step"]))
    if s["state"] == "fp32":
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        for name, x in (("m", m), ("v", torch.sqrt(v))):
            b = x.view(-1, 128)
            sf = (b.abs().amax(1) / 448).clamp(min=1e-30)
            s[name + "_s"].copy_(sf)
            s[name].copy_((b * (1 / sf)[:, None]).to(E4M3).view(-1).view(torch.uint8))
    s["p"].copy_(p)
    if "copy" in s:
        s["copy"].copy_(p)
    return _states(s)


# ------------------------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ------------------------------------------------------------------------------------------
#
# MXFP8 codes and scales and 8-bit states have no value here: a number next to the border of two codes (or a
# block's largest next to a border of its scale) goes to either side by the last bit of any 32-bit sum, a step
# of 1/16 that says nothing about the sum.  What they are rounded from is returned beside them where it is an
# output (ab, dprobs, the fp32 scales and the parameters).

def _decode(code, byte):
    return code.view(E4M3).to(F64) * torch.exp2(byte.to(F64) - 127).repeat_interleave(32, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in GLU:
        return _exact_glu(s, [int(k) for k in _counts(case, seed)])
    if op == "norm":
        x, y, w1, w2 = (s[k].to(F64) for k in ("x", "y", "post", "pre"))
        ry = 1 / torch.sqrt((y ** 2).mean(1) + s["eps"])
        z = (s["offset"] + w1) * (y * ry[:, None])
        if s["gate"] is not None:
            z *= s["gate"].to(F64)[:, None] if s["gate_kind"] == "token" else s["gate"].to(F64)
        r = s["x_scale"] * x + s["y_scale"] * z
        rr = 1 / torch.sqrt((r ** 2).mean(1) + s["eps"])
        return {"r": r, "n": (s["offset"] + w2) * (r * rr[:, None]), "rstd_y": ry, "rstd_r": rr}
    if op == "norm_grad":
        return _exact_norm_grad(s)
    b1, b2, k = s["beta1"], s["beta2"], s["step"]
    g = s["g"].to(F64) * s["grad_scale"].to(F64)
    if s["state"] == "fp32":
        m, v = s["m"].to(F64), s["v"].to(F64)
    else:
        m = s["m"].view(E4M3).to(F64) * s["m_s"].to(F64).repeat_interleave(128)
        v = (s["v"].view(E4M3).to(F64) * s["v_s"].to(F64).repeat_interleave(128)) ** 2
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g ** 2
    mean, square = m / (1 - b1 ** k), v / (1 - b2 ** k)
    p = s["p"].to(F64)
    p = p - s["lr"] * s["decay"] * p - s["lr"] * mean / (torch.sqrt(square) + s["eps"])
    out = {"p": p}
    if s["state"] == "fp32":
        out["m"], out["v"] = m, v
    else:
        for name, x in (("m", m), ("v", torch.sqrt(v))):
            out[name] = None
            out[name + "_s"] = (x.view(-1, 128).abs().amax(1) / 448).clamp(min=1e-30)
    if "copy" in s:
        out["copy"] = p
    return out


def _exact_glu(s, counts):
    e, t, rows, h, f = s["e"], s["t"], s["rows"], s["h"], s["f"]
    grad = s["op"] == "glu_grad"
    n = 2 * f if grad else f
    ab = torch.zeros((rows, 2 * f), dtype=F64, device=DEV)
    v = torch.zeros((rows, n), dtype=F64, device=DEV)
    dp = torch.zeros(rows, dtype=F64, device=DEV)
    first = 0
    for i, k in enumerate(counts):
        a_rows = slice(first, first + k)
        x = _decode(s["x"]["row_q"][a_rows], s["x"]["row_s"][:, a_rows].t().contiguous())
        p = s["probs"][a_rows].to(F64)[:, None]
        if grad:
            hp = (h + 127) // 128 * 128
            w = _decode(s["w"]["col_q"].view(e, f, hp)[i], s["w"]["col_s"].view(e, hp // 32, f)[i].t().contiguous())
            dh = x @ w[:, :h].t()
            a, b = s["ab"][a_rows].to(F64).chunk(2, 1)
            sg = torch.sigmoid(a)
            dp[a_rows] = (dh * b * a * sg).sum(1)
            v[a_rows] = torch.cat([dh * p * b * (sg + a * sg * (1 - sg)), dh * p * a * sg], 1)
        else:
            w = _decode(s["w"]["row_q"].view(e, 2 * f, h)[i], s["w"]["row_s"].view(h // 32, e, 2 * f)[:, i].t().contiguous())
            ab[a_rows] = x @ w.t()
            a, b = ab[a_rows].chunk(2, 1)
            v[a_rows] = p * b * a * torch.sigmoid(a)
        first += k
    out = {"y": v} if "y" in s else {"row_q": None, "row_s": None, "col_q": None, "col_s": None}
    if "ab" in s and not grad:
        out["ab"] = ab
    if grad:
        out["dprobs"] = dp
    return out


def _exact_norm_grad(s):
    """By the chain rule through each step of the forward, the statistics as given."""
    dn, dr, r, y = (s[k].to(F64) for k in ("dn", "dr", "r", "y"))
    rr, ry = s["rstd_r"].to(F64)[:, None], s["rstd_y"].to(F64)[:, None]
    w1, w2 = s["offset"] + s["post"].to(F64), s["offset"] + s["pre"].to(F64)
    c = r.shape[1]
    gate = None if s["gate"] is None else s["gate"].to(F64)[:, None] if s["gate_kind"] == "token" else s["gate"].to(F64)
    through = dn * w2 * rr - r * rr ** 3 * ((dn * w2 * r).sum(1, keepdim=True) / c)
    d = dr + through
    z = y * ry * w1
    dz = s["y_scale"] * d if gate is None else s["y_scale"] * d * gate
    dy = dz * w1 * ry - y * ry ** 3 * ((dz * w1 * y).sum(1, keepdim=True) / c)
    out = {"dx": s["x_scale"] * d, "dy": dy, "dpre_weight": (dn * r * rr).sum(0), "dpost_weight": (dz * y * ry).sum(0)}
    if gate is not None:
        out["dgate"] = (s["y_scale"] * d * z).sum(1 if s["gate_kind"] == "token" else 0)
    return out
