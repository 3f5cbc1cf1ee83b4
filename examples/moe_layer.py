"""A mixture-of-experts layer with a trained router, from end to end with this framework's kernels: norms around the
block, routing, tokens to their experts in MXFP8, both projections, back to the tokens, every gradient and an AdamW step.

    python examples/moe_layer.py [--tokens 4096 --hidden 1024 --ffn 512 --experts 32 --top-k 4 --steps 20 --keep 8bit]

The layer is norm(x + gate * sum_j p_j expert_j(norm(x))) over each token's top_k experts, p their softmax
probabilities over the sum of the chosen, with the usual loss that spreads the tokens over the experts.  What the backward
pass needs of the first projection is kept either in bf16, the gated projection being one kernel and the probabilities
applied where the rows return, or in 8 bits: then the activation takes the probabilities, and its gradient builds the
second projection's operand again.  It fits the output of a random layer of the same shape.  Torch multiplies by the
router's weight; everything else runs in libbsfp8.so.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp8_grouped_amd as bs  # noqa: E402

MX, ROW, COL, BOTH = bs.RECIPE_MX, bs.ROWWISE, bs.COLWISE, bs.ROWWISE | bs.COLWISE


class MoELayer:
    """fp32 master parameters, bf16 copies of the experts' weights that AdamW writes and the quantize reads."""

    def __init__(self, hidden, ffn, experts, top_k, keep="8bit", balance=0.01, seed=0, device="cuda"):
        if keep not in ("bf16", "8bit"):
            raise ValueError(f"keep: bf16 or 8bit, not {keep!r}")
        g = torch.Generator(device=device).manual_seed(seed)

        def rand(*shape, scale):
            return torch.randn(shape, generator=g, device=device) * scale

        self.h, self.f, self.e, self.k, self.dev = hidden, ffn, experts, top_k, device
        self.keep, self.balance = keep, balance
        self.router = rand(experts, hidden, scale=hidden ** -0.5)
        self.w1 = rand(experts * 2 * ffn, hidden, scale=hidden ** -0.5)  # each expert's a rows, then its b rows
        self.w2 = rand(experts * hidden, ffn, scale=ffn ** -0.5)
        # norm weights are kept as their distance from 1 (weight_offset), so that weight decay pulls them there
        self.pre, self.last = (torch.zeros(hidden, device=device) for _ in range(2))
        self.gate = torch.full((hidden,), 0.5, device=device)
        self.params = [self.router, self.w1, self.w2, self.pre, self.last, self.gate]
        self.w1c, self.w2c = self.w1.bfloat16(), self.w2.bfloat16()
        self.grads = [torch.zeros_like(p) for p in self.params]
        self.grouter, self.gw1, self.gw2, self.gpre, self.glast, self.ggate = self.grads
        self.s1 = torch.full((experts,), 2 * ffn, dtype=torch.int32, device=device)
        self.s2 = torch.full((experts,), hidden, dtype=torch.int32, device=device)
        self.q1 = bs.alloc_quantized(experts * 2 * ffn, hidden, experts, MX, BOTH, device)
        self.q2 = bs.alloc_quantized(experts * hidden, ffn, experts, MX, BOTH, device)
        self.quantize_weights()
        m, v = ([torch.zeros_like(p) for p in self.params] for _ in range(2))
        self.adamw = bs.adamw_plan(self.params, self.grads, m, v, None, None,
                                   copies=[None, self.w1c, self.w2c, None, None, None], decay_scales=[1, 1, 1, 0, 0, 0])
        self.step = 0

    def quantize_weights(self):
        bs.grouped_quantize(self.w1c, self.s1, MX, BOTH, self.q1)
        bs.grouped_quantize(self.w2c, self.s2, MX, BOTH, self.q2)

    def quantized(self, rows, cols, which=BOTH):
        return bs.alloc_quantized(rows, cols, self.e, MX, which, self.dev)

    def rows(self, rows, cols):
        return torch.empty((rows, cols), dtype=torch.bfloat16, device=self.dev)

    def forward(self, x):
        """x [T, h] bf16; a step's temporaries are kept for its backward."""
        T, R = x.shape[0], x.shape[0] * self.k
        first = bs.residual_norm(x, pre_weight=self.pre, weight_offset=1.0)
        n = first["n"]
        logits = n.float() @ self.router.t()
        score_sum = torch.empty(self.e, device=self.dev)
        route = bs.route_topk(logits, self.k, score_sum=score_sum)
        plan = bs.dispatch_plan(route["experts"], self.e, route["probs"])
        splits = plan["splits"]
        xq = bs.dispatch_quantize(n, plan, MX, BOTH, self.quantized(R, self.h))
        y = self.rows(R, self.h)
        if self.keep == "bf16":
            hidden = self.rows(R, 2 * self.f)
            hq = self.quantized(R, self.f)
            bs.grouped_gemm_swiglu(xq, self.h, self.q1, self.f, splits, R, ab=hidden, out=hq)
            bs.grouped_gemm_fprop(hq, self.f, self.q2, self.h, splits, R, y, bs.OUT_BF16)
            out = bs.combine(y, plan, weights=route["probs"])
        else:
            h = self.rows(R, 2 * self.f)
            bs.grouped_gemm_fprop(xq, self.h, self.q1, 2 * self.f, splits, R, h, bs.OUT_BF16)
            hq, hidden = self.quantized(R, self.f, ROW), self.quantized(R, 2 * self.f, ROW)
            bs.grouped_act_checkpoint(bs.ACT_SWIGLU, h, splits, MX, ROW, hq, hidden, probs=plan["probs"])
            bs.grouped_gemm_fprop(hq, self.f, self.q2, self.h, splits, R, y, bs.OUT_BF16)
            out = bs.combine(y, plan)
            hq = y = None  # (the gradient builds hq's other layout again)
        last = bs.residual_norm(x, out, pre_weight=self.last, gate=self.gate, gate_kind=bs.GATE_CHANNEL, weight_offset=1.0)
        # e * sum over the experts of their share of the choices and their mean score: 1 where the tokens are spread evenly
        self.balance_loss = (splits.float() * score_sum).sum() * (self.e / (R * T))
        self.kept = (x, first, logits, route, plan, xq, hidden, hq, y, out, last)
        return last["n"]

    def backward(self, dout):
        """From dout [T, h] bf16: the parameters' gradients (with balance * balance_loss) and that of x."""
        x, first, logits, route, plan, xq, hidden, hq, y, out, last = self.kept
        T, R, splits = x.shape[0], x.shape[0] * self.k, plan["splits"]
        d = bs.residual_norm_grad(dout, None, last["r"], last["rstd_r"], self.last, y=out, gate=self.gate,
                                  gate_kind=bs.GATE_CHANNEL, weight_offset=1.0, dpre_weight=self.glast, dgate=self.ggate)
        if self.keep == "bf16":
            dprobs = bs.combine_grad(d["dy"], plan, y=y, weights=route["probs"], dy=False)["dweights"]
            dy = bs.dispatch_quantize(d["dy"], plan, MX, BOTH, self.quantized(R, self.h), weights=route["probs"])
            dh = self.quantized(R, 2 * self.f)
            bs.grouped_gemm_swiglu_grad(dy, self.h, self.q2, self.f, hidden, splits, R, out=dh)
        else:
            dy = bs.dispatch_quantize(d["dy"], plan, MX, BOTH, self.quantized(R, self.h))
            da = self.rows(R, self.f)
            bs.grouped_gemm_dgrad(dy, self.h, self.q2, self.f, splits, R, da, bs.OUT_BF16)
            dh, hq = self.quantized(R, 2 * self.f), self.quantized(R, self.f, COL)
            drows = torch.empty(R, device=self.dev)
            bs.grouped_act_checkpoint_grad(bs.ACT_SWIGLU, hidden, da, splits, MX, BOTH, dh, probs=plan["probs"], y=hq,
                                           dprobs=drows)
            # the rows' numbers at their choices: weights' gradient of one channel, whose dout is 1
            dprobs = torch.empty((T, self.k), device=self.dev)
            ones = torch.ones((T, 1), device=self.dev)
            bs.combine_grad(ones, plan, y=drows.view(R, 1), dy=False, dweights=dprobs)
        bs.grouped_gemm_wgrad(dy, self.h, hq, self.f, splits, R, MX, self.gw2.view(self.e, self.h, self.f))
        bs.grouped_gemm_wgrad(dh, 2 * self.f, xq, self.h, splits, R, MX, self.gw1.view(self.e, 2 * self.f, self.h))
        dx = self.rows(R, self.h)
        bs.grouped_gemm_dgrad(dh, 2 * self.f, self.q1, self.h, splits, R, dx, bs.OUT_BF16)
        dscores = splits.float() * (self.balance * self.e / (R * T))
        dlogits = bs.route_topk_grad(dprobs, logits, route["experts"], bs.ROUTE_SOFTMAX, True, 1.0, dscore_sum=dscores)
        torch.mm(dlogits.t(), first["n"].float(), out=self.grouter)
        dn = bs.combine(dx, plan, add=(dlogits @ self.router).bfloat16())
        return bs.residual_norm_grad(dn, d["dx"], first["r"], first["rstd_r"], self.pre, weight_offset=1.0,
                                     dpre_weight=self.gpre)["dx"]

    def update(self, lr, **more):
        self.step += 1
        bs.adamw_step(self.adamw, lr, step=self.step, **more)
        self.quantize_weights()


def train(tokens=4096, hidden=1024, ffn=512, experts=32, top_k=4, steps=20, keep="8bit", lr=3e-3, seed=0, log=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    teacher, layer = (MoELayer(hidden, ffn, experts, top_k, keep, seed=seed + 1 + i) for i in range(2))
    losses = []
    for i in range(steps):
        x = torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16()
        target = teacher.forward(x).float()
        torch.cuda.synchronize()
        t = time.time()
        miss = layer.forward(x).float() - target
        layer.backward((miss * (2.0 / tokens)).bfloat16())
        layer.update(lr, beta2=0.99, weight_decay=0.0)
        losses.append(miss.square().mean())
        torch.cuda.synchronize()
        if log:
            log(f"step {i + 1}: loss {float(losses[-1]):.5f}  balance {float(layer.balance_loss):.3f}  "
                f"{1e3 * (time.time() - t):.2f} ms")
    return [float(v) for v in losses]


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 4096), ("hidden", 1024), ("ffn", 512), ("experts", 32), ("top-k", 4), ("steps", 20)):
        p.add_argument("--" + name, type=int, default=default)
    p.add_argument("--keep", choices=["bf16", "8bit"], default="8bit")
    p.add_argument("--lr", type=float, default=3e-3)
    a = p.parse_args()
    train(a.tokens, a.hidden, a.ffn, a.experts, a.top_k, a.steps, a.keep, a.lr, log=lambda m: print(m, flush=True))


if __name__ == "__main__":
    main()
