"""The operators that bring tokens to their experts and back, and that keep an expert layer's activations for its
gradient, as cases that can be timed and compared: the router's choice of experts and its gradient, the sort of the
choices by expert, the rows gathered for the experts' products (as they are, or straight into MXFP8), the weighted sum
back and its gradient, and the activation between two projections with its input kept in 8 bits, and its gradient.

`run` computes a case in plain torch operations, or, where `own` is true, with this framework's kernels.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3, E8M0, BF16, F32, F64 = torch.float8_e4m3fn, torch.float8_e8m0fnu, torch.bfloat16, torch.float32, torch.float64
I32 = torch.int32
NONE = float("-inf")


# ------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------

def listed():
    return [
        # serving: four tokens choose 8 of 128 experts by sigmoid scores with a selection bias
        {"name": "route_tokens", "op": "route", "tokens": 4, "experts": 128, "top_k": 8, "type": "bf16",
         "scoring": "sigmoid", "bias": True, "renormalize": True, "masked": 0.0, "sum": False},
        # a training step's router over 131072 tokens, with the scores' sums for a load-balancing loss, and its gradient
        {"name": "route_layer", "op": "route", "tokens": 131072, "experts": 128, "top_k": 8, "type": "fp32",
         "scoring": "softmax", "bias": False, "renormalize": True, "masked": 0.0, "sum": True},
        {"name": "route_grad_layer", "op": "route_grad", "tokens": 131072, "experts": 128, "top_k": 8, "type": "fp32",
         "scoring": "softmax", "bias": False, "renormalize": True, "masked": 0.0, "sum": True},
        # the choices of the same tokens sorted by expert
        {"name": "plan_tokens", "op": "plan", "tokens": 4, "experts": 128, "top_k": 8, "dropped": 0.0},
        {"name": "plan_layer", "op": "plan", "tokens": 131072, "experts": 128, "top_k": 8, "dropped": 0.0},
        # serving: four tokens' rows for their experts, quantized for the gated projection
        {"name": "dispatch_tokens", "op": "dispatch", "tokens": 4, "experts": 128, "top_k": 8, "cols": 7168,
         "dropped": 0.0, "weighted": False, "out": "mxfp8_row"},
        # training: the rows of an expert layer quantized in both layouts, for its products and its weight gradient
        {"name": "dispatch_layer", "op": "dispatch", "tokens": 16384, "experts": 32, "top_k": 4, "cols": 4096,
         "dropped": 0.0, "weighted": False, "out": "mxfp8"},
        # the experts' results summed back: four tokens, and a layer on top of its residual stream
        {"name": "combine_tokens", "op": "combine", "tokens": 4, "experts": 128, "top_k": 8, "cols": 7168,
         "dropped": 0.0, "weighted": True, "add": False, "type": "bf16"},
        {"name": "combine_layer", "op": "combine", "tokens": 16384, "experts": 32, "top_k": 4, "cols": 4096,
         "dropped": 0.0, "weighted": True, "add": True, "type": "bf16"},
        # its gradient on a ragged step whose padding tokens (a tenth) go to no expert
        {"name": "combine_grad_odd", "op": "combine_grad", "tokens": 16411, "experts": 32, "top_k": 3, "cols": 2050,
         "dropped": 0.1, "weighted": True, "add": False, "type": "bf16"},
        # squared ReLU between two projections, fc1's output kept in 8 bits, on few experts and a padded buffer
        {"name": "act_odd", "op": "act", "act": "srelu", "rows": 4099, "pad": 61, "experts": 8, "ffn": 4128},
        # the gradient of a gated layer from its 8-bit checkpoint
        {"name": "act_grad_layer", "op": "act_grad", "act": "swiglu", "rows": 65536, "pad": 0, "experts": 32,
         "ffn": 2048},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["route", "route_grad", "plan", "dispatch", "combine", "combine_grad", "act", "act_grad"])
    if op in ("act", "act_grad"):
        return {"op": op, "act": rng.choice(["srelu", "swiglu"]), "rows": log(1, 32768),
                "pad": rng.choice([0, rng.randint(1, 300)]), "experts": log(1, 64), "ffn": 32 * log(4, 64)}
    experts = log(2, 256)
    top_k = min(experts, rng.choice([1, 2, 3, 4, 6, 8]))
    c = {"op": op, "tokens": log(1, 65536), "experts": experts, "top_k": top_k}
    if op in ("route", "route_grad"):
        c |= {"type": rng.choice(["fp32", "bf16"]), "scoring": rng.choice(["softmax", "sigmoid"]),
              "bias": rng.random() < 0.5, "renormalize": rng.random() < 0.7, "masked": rng.choice([0.0, 0.1]),
              "sum": rng.random() < 0.5}
        return c
    c["dropped"] = rng.choice([0.0, 0.0, 0.2])
    if op == "plan":
        return c
    # (tokens that keep a drawn case within the largest listed one)
    c["cols"] = log(64, 7168)
    c["tokens"] = min(c["tokens"], max(1, (1 << 26) // (c["cols"] * top_k)))
    c["weighted"] = rng.random() < 0.5
    if op == "dispatch":
        c["out"] = rng.choice(["bf16", "fp32", "mxfp8", "mxfp8_row"])
        if c["out"].startswith("mxfp8"):
            c["cols"] = (c["cols"] + 31) // 32 * 32
        return c
    c |= {"add": op == "combine" and rng.random() < 0.5, "type": rng.choice(["bf16", "fp32"])}
    return c


def _dtype(name):
    return {"fp32": F32, "bf16": BF16}[name]


def work(case):
    op = case["op"]
    q = 33 / 32  # bytes of an MXFP8 value with its share of the scale
    if op in ("act", "act_grad"):
        n = case["rows"] * case["ffn"]
        wide = n * (2 if case["act"] == "swiglu" else 1)  # fc1's output
        if op == "act":
            return {"bytes": 2 * wide + q * wide + 2 * q * n + 4 * case["rows"], "flops": 12 * n}
        return {"bytes": q * wide + 2 * n + 2 * q * wide + q * n + 8 * case["rows"], "flops": 30 * n}
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    if op in ("route", "route_grad"):
        size = 2 if case["type"] == "bf16" else 4
        more = 4 * e * (int(case["bias"]) + int(case["sum"]))
        return {"bytes": t * e * size * (1 if op == "route" else 2) + 8 * t * k + more, "flops": 10 * t * e}
    if op == "plan":
        return {"bytes": 20 * t * k + 4 * e, "flops": 4 * t * k}
    c = case["cols"]
    live = t * k * (1 - case["dropped"])
    weights = 4 * t * k if case["weighted"] else 0
    if op == "dispatch":
        out, size = {"bf16": (2, 2), "fp32": (4, 4), "mxfp8": (2 * q, 2), "mxfp8_row": (q, 2)}[case["out"]]
        return {"bytes": t * c * size + live * c * out + 4 * t * k + weights, "flops": 2 * live * c}
    size = 2 if case["type"] == "bf16" else 4
    if op == "combine":
        return {"bytes": live * c * size + t * c * size * (2 if case["add"] else 1) + 4 * t * k + weights,
                "flops": 2 * live * c}
    # (without weights the gradient is a copy of dout's rows and reads no y)
    return {"bytes": t * c * size + live * c * size * (2 if case["weighted"] else 1) + 4 * t * k + 2 * weights,
            "flops": 3 * live * c}


# ------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------

def _randn(shape, g, scale=1.0):
    return torch.randn(shape, generator=g, device=DEV, dtype=F32) * scale


def _rand(shape, g):
    return torch.rand(shape, generator=g, device=DEV, dtype=F32)


def _routing(case, g):
    """Experts of each token, without repetition, some experts more popular than others; tokens that are dropped
    (padding) have none."""
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    liking = _randn((t, e), g) + _randn((e,), g)
    experts = liking.topk(k, 1).indices.to(I32)
    experts[_rand((t,), g) < case["dropped"]] = -1
    return experts


def _plan(experts, num_experts, probs):
    """The choices t * top_k + j sorted by expert: rows per expert, each choice's row (-1 where it has no expert), each
    row's choice (-1 past the last) and its probability (0)."""
    e = experts.reshape(-1).long()
    e = torch.where((e >= 0) & (e < num_experts), e, num_experts)
    count = torch.zeros(num_experts + 1, dtype=torch.long, device=DEV).index_add_(0, e, torch.ones_like(e))[:num_experts]
    order = torch.sort(e, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(e.numel(), device=DEV)
    dropped = e == num_experts
    out = {"splits": count.to(I32), "rows": torch.where(dropped, -1, place).to(I32).view(experts.shape),
           "choices": torch.where(dropped[order], -1, order).to(I32)}
    if probs is not None:
        out["probs"] = torch.where(dropped[order], 0, probs.reshape(-1)[order])
    return out


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op in ("act", "act_grad"):
        rows, f, e = case["rows"], case["ffn"], case["experts"]
        wide = f * (2 if case["act"] == "swiglu" else 1)
        share = torch.softmax(_randn((e,), g), 0).cumsum(0)
        of = torch.bucketize(_rand((rows,), g), share).clamp(max=e - 1)
        s["splits"] = torch.zeros(e, dtype=torch.long, device=DEV).index_add_(0, of, torch.ones_like(of)).to(I32)
        s["of"] = torch.sort(of).values
        s["cap"] = cap = rows + case["pad"]
        s["probs"] = _rand((cap,), g)
        # rows past the last expert's hold any bits
        h = torch.full((cap, wide), float("nan"), dtype=BF16, device=DEV)
        h[:rows] = _randn((rows, wide), g).to(BF16)
        bound = 128 * ((cap + 127 * e) // 128)

        def layouts(n, row=True, col=True):
            q = {}
            if row:
                q["row_q"] = torch.zeros((cap, n), dtype=torch.uint8, device=DEV)
                q["row_s"] = torch.zeros((n // 32, cap), dtype=torch.uint8, device=DEV)
            if col:
                q["col_q"] = torch.zeros(n * bound, dtype=torch.uint8, device=DEV)
                q["col_s"] = torch.zeros(n * bound // 32, dtype=torch.uint8, device=DEV)
            return q

        if op == "act":
            s["h"], s["q"], s["kept"] = h, layouts(f), layouts(wide, col=False)
            return s
        s["kept"] = layouts(wide, col=False)
        codes, scale = _mx(h[:rows].float())
        s["kept"]["row_q"][:rows] = codes
        s["kept"]["row_s"][:, :rows] = scale.t()
        s["dy"] = torch.full((cap, f), float("nan"), dtype=BF16, device=DEV)
        s["dy"][:rows] = _randn((rows, f), g, 0.01).to(BF16)
        s["q"], s["y"], s["dprobs"] = layouts(wide), layouts(f, row=False), torch.zeros(cap, dtype=F32, device=DEV)
        return s
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    if op in ("route", "route_grad"):
        l = _randn((t, e), g, 1.5) + _randn((e,), g, 0.5)
        # experts that a token may not choose, and padding tokens that choose none
        l[_rand((t, e), g) < case["masked"]] = NONE
        l[_rand((t,), g) < case["masked"]] = NONE
        s["logits"] = l.to(_dtype(case["type"]))
        s["bias_of"] = _randn((e,), g, 0.1) if case["bias"] else None
        s["scale"] = 2.5 if case["scoring"] == "sigmoid" else 1.0
        if op == "route_grad":
            s["chosen"] = _choose(s)
            s["dprobs"] = _randn((t, k), g, 0.01)
            s["dsum"] = _randn((e,), g, 0.001) if case["sum"] else None
        return s
    experts, probs = _routing(case, g), _rand((t, k), g)
    if op == "plan":
        return s | {"chosen": experts, "probs": probs}
    plan = _plan(experts, e, None)
    n, c = t * k, case["cols"]
    s |= {"plan": plan, "weights": probs if case["weighted"] else None}
    if op == "dispatch":
        x = _randn((t, c), g)
        if not case["out"].startswith("mxfp8"):
            s["x"] = x.to(_dtype(case["out"]))
            s["to"] = torch.zeros((n, c), dtype=s["x"].dtype, device=DEV)
            return s
        s["x"] = x.to(BF16)
        s["q"] = {"row_q": torch.zeros((n, c), dtype=torch.uint8, device=DEV),
                  "row_s": torch.zeros((c // 32, n), dtype=torch.uint8, device=DEV)}
        if case["out"] == "mxfp8":
            bound = 128 * ((n + 127 * e) // 128)
            s["q"]["col_q"] = torch.zeros(c * bound, dtype=torch.uint8, device=DEV)
            s["q"]["col_s"] = torch.zeros(c * bound // 32, dtype=torch.uint8, device=DEV)
        return s
    kind = _dtype(case["type"])
    s["y"] = _randn((n, c), g).to(kind)
    if op == "combine":
        s["added"] = _randn((t, c), g, 3.0).to(kind) if case["add"] else None
        return s
    s["dout"] = _randn((t, c), g, 0.01).to(kind)
    s["dy"] = torch.zeros((n, c), dtype=kind, device=DEV)
    return s


# ------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)(s)


def _shown(q, name=""):
    """MXFP8 layouts as the values that their codes and scales stand for."""
    return {name + k: v.view(E4M3 if k.endswith("_q") else E8M0) for k, v in q.items()}


def _own(s):
    import block_scaled_fp8_grouped_amd as bs

    op = s["op"]
    if op in ("act", "act_grad"):
        act = bs.ACT_SRELU if s["act"] == "srelu" else bs.ACT_SWIGLU
        if op == "act":
            bs.grouped_act_checkpoint(act, s["h"], s["splits"], bs.RECIPE_MX, bs.ROWWISE | bs.COLWISE, s["q"], s["kept"],
                                      probs=s["probs"])
            return _shown(s["q"]) | _shown(s["kept"], "kept_")
        bs.grouped_act_checkpoint_grad(act, s["kept"], s["dy"], s["splits"], bs.RECIPE_MX, bs.ROWWISE | bs.COLWISE, s["q"],
                                       probs=s["probs"], y=s["y"], dprobs=s["dprobs"])
        return _shown(s["q"]) | _shown(s["y"], "y_") | {"dprobs": s["dprobs"]}
    if op in ("route", "route_grad"):
        how = dict(scoring=bs.ROUTE_SOFTMAX if s["scoring"] == "softmax" else bs.ROUTE_SIGMOID,
                   renormalize=s["renormalize"], scale=s["scale"])
        if op == "route":
            total = torch.empty(s["experts"], dtype=F32, device=DEV) if s["sum"] else None
            return bs.route_topk(s["logits"], s["top_k"], bias=s["bias_of"], score_sum=total, **how)
        return bs.route_topk_grad(s["dprobs"], s["logits"], s["chosen"], dscore_sum=s["dsum"], **how)
    if op == "plan":
        return bs.dispatch_plan(s["chosen"], s["experts"], probs=s["probs"])
    if op == "dispatch":
        if "to" in s:
            return bs.dispatch(s["x"], s["plan"], weights=s["weights"], out=s["to"])
        which = bs.ROWWISE | (bs.COLWISE if "col_q" in s["q"] else 0)
        return _shown(bs.dispatch_quantize(s["x"], s["plan"], bs.RECIPE_MX, which, s["q"], weights=s["weights"]))
    if op == "combine":
        return bs.combine(s["y"], s["plan"], weights=s["weights"], add=s["added"])
    return bs.combine_grad(s["dout"], s["plan"], y=s["y"] if s["weighted"] else None, weights=s["weights"], dy=s["dy"])


def _mx(v):
    """MXFP8 of fp32 blocks of 32 along the last axis: e4m3 codes and E8M0 bytes."""
    b = v.unflatten(-1, (-1, 32))
    frac, e = torch.frexp(b.abs().amax(-1))
    e = torch.where(frac == 0, -127, (e - 9 + (frac > 0.875)).clamp(-127, 127))
    codes = (b * torch.exp2(-e.to(F32)).unsqueeze(-1)).to(E4M3).view(torch.uint8)
    return codes.flatten(-2), (e + 127).to(torch.uint8)


def _values(codes, scale):
    """fp32 values of e4m3 codes [..., n] and E8M0 bytes [..., n / 32]."""
    two = torch.exp2(scale.to(F32) - 127)
    return (codes.view(E4M3).to(F32).unflatten(-1, (-1, 32)) * two.unsqueeze(-1)).flatten(-2)


def _columns(q, v, of, splits):
    """The layout whose blocks run along each expert's rows: v [live, n] with the rows' experts."""
    k = splits.long()
    kp = (k + 127) // 128 * 128
    live, n = v.shape
    at = (kp.cumsum(0) - kp - k.cumsum(0) + k)[of] + torch.arange(live, device=DEV)
    bound = q["col_q"].numel() // n
    tall = torch.zeros((n, bound), dtype=F32, device=DEV)
    tall[:, at] = v.t()
    codes, scale = _mx(tall)
    q["col_s"].view(-1, n).copy_(scale.t())
    # an expert's part begins at n times its first row; a channel's codes lie side by side in it
    first = kp.cumsum(0) - kp
    place = ((n - 1) * first[of] + at)[:, None] + torch.arange(n, device=DEV) * kp[of][:, None]
    q["col_q"][place] = codes[:, at].t()


def _quantized(q, v, of, splits):
    live = v.shape[0]
    if "row_q" in q:
        codes, scale = _mx(v)
        q["row_q"][:live] = codes
        q["row_s"][:, :live] = scale.t()
    if "col_q" in q:
        _columns(q, v, of, splits)


def _exp2(x):
    """2^x in 32 bits by steps that give the same bits everywhere: 2^floor(x + 1/2) times a Taylor polynomial."""
    x = x.clamp(-126, 126)
    k = torch.floor(x + 0.5)
    r = x - k
    p = 1.52527338e-05 * r + 0.000154035304
    p = p * r + 0.00133335581
    p = p * r + 0.00961812911
    p = p * r + 0.0555041087
    p = p * r + 0.240226507
    p = p * r + 0.693147182
    p = p * r + 1.0
    return p * ((k.to(I32) + 127) << 23).view(F32)


def _sigmoid(x):
    return 1 / (1 + _exp2(x * -1.44269502))


def _scores(l, scoring):
    out = torch.isneginf(l)
    if scoring == "sigmoid":
        return torch.where(out, 0, _sigmoid(l))
    p = torch.exp(l - torch.where(out.all(1), 0, l.amax(1))[:, None])
    return p / torch.where(out.all(1), 1, p.sum(1))[:, None]


def _choose(s):
    """The experts of the largest keys, the lowest index first among equals, -1 where no other is left."""
    l = s["logits"].float()
    key = l if s["scoring"] == "softmax" else _scores(l, "sigmoid")
    if s["bias_of"] is not None:
        key = key + s["bias_of"]
    key = torch.where(torch.isneginf(l), NONE, key)
    best, at = torch.sort(key, dim=1, descending=True, stable=True)
    return torch.where(torch.isneginf(best), -1, at)[:, :s["top_k"]].to(I32)


def _of_chosen(l, s, chosen):
    """The chosen experts' scores (0 for none) and what they are divided by."""
    none, at = chosen < 0, chosen.long().clamp(min=0)
    if s["renormalize"]:
        mine = l.gather(1, at)
        if s["scoring"] == "softmax":
            p = torch.exp(mine - torch.where(none, NONE, mine).amax(1).nan_to_num(neginf=0)[:, None])
        else:
            p = _sigmoid(mine)
        p = torch.where(none, 0, p)
        return p, torch.where(none.all(1), 1, p.sum(1))[:, None]
    return torch.where(none, 0, _scores(l, s["scoring"]).gather(1, at)), 1.0


def _plain_route(s):
    l = s["logits"].float()
    if s["op"] == "route":
        chosen = _choose(s)
        p, by = _of_chosen(l, s, chosen)
        out = {"probs": p / by * s["scale"], "experts": chosen}
        if s["sum"]:
            out["score_sum"] = _scores(l, s["scoring"]).sum(0, dtype=F64).to(F32)
        return out
    chosen, dp = s["chosen"], s["dprobs"] * s["scale"]
    p, by = _of_chosen(l, s, chosen)
    at = chosen.long().clamp(min=0)
    part = p / by
    scores = _scores(l, s["scoring"])
    d = torch.zeros_like(l)
    if s["renormalize"]:
        mine = part * (dp - (dp * part).sum(1, keepdim=True))
        mine = mine if s["scoring"] == "softmax" else mine * (1 - p)
        d.scatter_add_(1, at, torch.where(chosen < 0, 0, mine))
        back = torch.zeros_like(l)
    else:
        back = torch.zeros_like(l).scatter_add_(1, at, torch.where(chosen < 0, 0, dp))
    if s["dsum"] is not None:
        back = back + s["dsum"]
    if s["scoring"] == "softmax":
        d = d + scores * (back - (back * scores).sum(1, keepdim=True))
    else:
        d = d + back * scores * (1 - scores)
    return d.to(s["logits"].dtype)



def _plain_act(s):
    n, f = s["rows"], s["ffn"]
    p = s["probs"][:n, None]
    if s["op"] == "act":
        h = s["h"][:n].float()
    else:
        h = _values(s["kept"]["row_q"][:n], s["kept"]["row_s"][:, :n].t())
        dy = s["dy"][:n].float()
    if s["act"] == "srelu":
        r = h.clamp(min=0)
        value = r * r
    else:
        a, b = h[:, :f], h[:, f:]
        sg = _sigmoid(a)
        value = (a * sg) * b
    of = s["of"]
    if s["op"] == "act":
        _quantized(s["q"], value * p, of, s["splits"])
        codes, scale = _mx(h)
        s["kept"]["row_q"][:n] = codes
        s["kept"]["row_s"][:, :n] = scale.t()
        return _shown(s["q"]) | _shown(s["kept"], "kept_")
    if s["act"] == "srelu":
        back = ((2 * r) * p) * dy
    else:
        q = dy * p
        back = torch.cat([(q * b) * (sg * (1 + a * (1 - sg))), q * (a * sg)], 1)
    _quantized(s["q"], back, of, s["splits"])
    _quantized(s["y"], value * p, of, s["splits"])
    s["dprobs"][:n] = (dy * value).sum(1)
    return _shown(s["q"]) | _shown(s["y"], "y_") | {"dprobs": s["dprobs"]}


def _plain(s):
    op = s["op"]
    if op in ("act", "act_grad"):
        return _plain_act(s)
    if op in ("route", "route_grad"):
        return _plain_route(s)
    if op == "plan":
        return _plan(s["chosen"], s["experts"], s["probs"])
    k, w, rows = s["top_k"], s["weights"], s["plan"]["rows"].long()
    if op == "dispatch":
        choices = s["plan"]["choices"].long()
        at = choices[choices >= 0]
        v = s["x"][at // k].float()
        if w is not None:
            v = v * w.reshape(-1)[at][:, None]
        if "to" in s:
            s["to"][:v.shape[0]] = v.to(s["to"].dtype)
            return s["to"]
        k = s["plan"]["splits"].long()
        of = torch.repeat_interleave(torch.arange(s["experts"], device=DEV), k, output_size=v.shape[0])
        _quantized(s["q"], v, of, s["plan"]["splits"])
        return _shown(s["q"])
    here = rows >= 0
    if op == "combine":
        each = s["y"][rows.clamp(min=0)].float()
        each = torch.where(here[:, :, None], each if w is None else each * w[:, :, None], 0)
        total = each.sum(1)
        return (total if s["added"] is None else s["added"].float() + total).to(s["y"].dtype)
    dout = s["dout"].float()
    token, slot = here.nonzero(as_tuple=True)
    at = rows[token, slot]
    back = dout[token]
    out = {"dy": s["dy"]}
    if w is not None:
        out["dweights"] = torch.zeros_like(w)
        out["dweights"][token, slot] = (back * s["y"][at].float()).sum(1)
        back = back * w[token, slot][:, None]
    s["dy"][at] = back.to(s["dy"].dtype)
    return out


# ------------------------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ------------------------------------------------------------------------------------------
#
# MXFP8 codes of computed values (an activation, a weighted row) have no value here: a number next to the border of
# two codes, or a block's largest next to a border of its scale, goes to either side by the last bit of any 32-bit
# value.  Codes of values that are inputs do.  Experts are whole numbers and are compared as such.

def _codes64(v):
    """Code values and scales of MXFP8 blocks along the last axis, by their definition: the least power of two that
    brings the block's largest to 448 at most, and the nearest of e4m3's numbers."""
    b = v.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    e = torch.where(top > 0, torch.ceil(torch.log2(top / 448)), -127.0)
    e = torch.where(top > 448 * torch.exp2(e), e + 1, torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e)).clamp(min=-127)
    x = b * torch.exp2(-e).unsqueeze(-1)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).flatten(-2), torch.exp2(e)


def _rows64(v, cap):
    codes, scale = _codes64(v)
    q = torch.zeros((cap, v.shape[1]), dtype=F64, device=DEV)
    q[:v.shape[0]] = codes
    # a byte of 0, as the buffers hold it before, stands for 2^-127
    sc = torch.full((v.shape[1] // 32, cap), 2.0 ** -127, dtype=F64, device=DEV)
    sc[:, :v.shape[0]] = scale.t()
    return q, sc


def _exact_route(s):
    l = s["logits"].to(F64)
    t, k = l.shape[0], s["top_k"]
    chosen = _choose(s) if s["op"] == "route" else s["chosen"]
    l = l.requires_grad_()
    open_ = ~torch.isneginf(s["logits"])
    safe = torch.where(open_, l, 0.0)
    if s["scoring"] == "softmax":
        top = torch.where(open_, safe, -1e30).amax(1, keepdim=True).detach()
        weight = torch.where(open_, torch.exp(safe - top), 0.0)
        scores = weight / weight.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        scores = torch.where(open_, torch.sigmoid(safe), 0.0)
    mine = torch.where(chosen >= 0, scores.gather(1, chosen.long().clamp(min=0)), 0.0)
    if s["renormalize"]:
        mine = mine / mine.sum(1, keepdim=True).clamp(min=1e-300)
    probs, total = s["scale"] * mine, scores.sum(0)
    if s["op"] == "route":
        out = {"probs": probs.detach(), "experts": None}
        return out | ({"score_sum": total.detach()} if s["sum"] else {})
    loss = (probs * s["dprobs"].to(F64)).sum()
    if s["dsum"] is not None:
        loss = loss + (total * s["dsum"].to(F64)).sum()
    loss.backward()
    return l.grad


def _exact_act(s):
    n, f, cap = s["rows"], s["ffn"], s["cap"]
    if s["op"] == "act":
        q, sc = _rows64(s["h"][:n].to(F64), cap)
        return {"row_q": None, "row_s": None, "col_q": None, "col_s": None, "kept_row_q": q, "kept_row_s": sc}
    step = torch.exp2(s["kept"]["row_s"][:, :n].t().to(F64) - 127).repeat_interleave(32, 1)
    h = s["kept"]["row_q"][:n].view(E4M3).to(F64) * step
    if s["act"] == "srelu":
        value = torch.relu(h) ** 2
    else:
        value = h[:, :f] * torch.sigmoid(h[:, :f]) * h[:, f:]
    dprobs = torch.zeros(cap, dtype=F64, device=DEV)
    dprobs[:n] = (value * s["dy"][:n].to(F64)).sum(1)
    none = dict.fromkeys(["row_q", "row_s", "col_q", "col_s", "y_col_q", "y_col_s"])
    return none | {"dprobs": dprobs}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("act", "act_grad"):
        return _exact_act(s)
    if op in ("route", "route_grad"):
        return _exact_route(s)
    if op == "plan":
        # a choice's row is the number of choices that come before it; a row past the last has the probability 0
        e = s["chosen"].reshape(-1).cpu()
        probs = s["probs"].reshape(-1).to(F64).cpu()
        parts = [probs[e == i] for i in range(case["experts"])]
        live = torch.cat(parts)
        return {"splits": None, "rows": None, "choices": None,
                "probs": torch.cat([live, torch.zeros(e.numel() - live.numel(), dtype=F64)]).to(DEV)}
    k, choices = case["top_k"], s["plan"]["choices"].long()
    token, w = choices // k, s["weights"]
    live = int((choices >= 0).sum())
    if op == "dispatch":
        if "to" in s:
            out = torch.zeros(s["to"].shape, dtype=F64, device=DEV)
            out[:live] = s["x"].to(F64)[token[:live]]
            if w is not None:
                out[:live] *= w.reshape(-1).to(F64)[choices[:live]][:, None]
            return out
        if w is not None:
            return None
        out = dict.fromkeys(s["q"])
        out["row_q"], out["row_s"] = _rows64(s["x"].to(F64)[token[:live]], choices.numel())
        return out
    y = s["y"].to(F64)
    if op == "combine":
        weight = torch.ones(live, dtype=F64, device=DEV) if w is None else w.reshape(-1).to(F64)[choices[:live]]
        total = torch.zeros((case["tokens"], case["cols"]), dtype=F64, device=DEV)
        total.index_add_(0, token[:live], y[:live] * weight[:, None])
        return total if s["added"] is None else total + s["added"].to(F64)
    back = s["dout"].to(F64)[token[:live]]
    out = {"dy": torch.zeros(s["dy"].shape, dtype=F64, device=DEV)}
    if w is None:
        out["dy"][:live] = back
        return out
    out["dy"][:live] = back * w.reshape(-1).to(F64)[choices[:live]][:, None]
    dw = torch.zeros(w.numel(), dtype=F64, device=DEV)
    dw[choices[:live]] = (back * y[:live]).sum(1)
    return out | {"dweights": dw.view_as(w)}
