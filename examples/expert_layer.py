"""One expert layer trained from end to end with this framework's kernels: norms around the block, MXFP8
quantize, gated projection, second projection, their gradients and an AdamW step over all parameters.

    python examples/expert_layer.py [--tokens 4096 --hidden 1024 --ffn 512 --experts 8 --steps 20 --state 8bit]

The layer is norm(x + gate * experts(norm(x))), each token at one expert, weighted by its routing
probability (the router itself is not trained here: the routes are given); the residual sum, its gate and the
norm of the next block are one kernel.  It fits the output of a random layer of the same shape.  Torch sorts the tokens by expert; everything else runs in libbsfp8.so.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp8_grouped_amd as bs  # noqa: E402

MX, ROW, COL, BOTH = bs.RECIPE_MX, bs.ROWWISE, bs.COLWISE, bs.ROWWISE | bs.COLWISE


class ExpertLayer:
    """fp32 master parameters, bf16 copies of the experts' weights that AdamW writes and the quantize reads."""

    def __init__(self, hidden, ffn, experts, state="8bit", seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def rand(*shape, scale):
            return torch.randn(shape, generator=g, device=device) * scale

        self.h, self.f, self.e, self.dev, self.seed = hidden, ffn, experts, device, seed
        self.w1 = rand(experts * 2 * ffn, hidden, scale=hidden ** -0.5)  # each expert's a rows, then its b rows
        self.w2 = rand(experts * hidden, ffn, scale=ffn ** -0.5)
        # norm weights are kept as their distance from 1 (weight_offset), so that weight decay pulls them there
        self.pre, self.last = (torch.zeros(hidden, device=device) for _ in range(2))
        self.gate = torch.full((hidden,), 0.5, device=device)
        self.params = [self.w1, self.w2, self.pre, self.last, self.gate]
        self.w1c, self.w2c = self.w1.bfloat16(), self.w2.bfloat16()
        self.grads = [torch.zeros_like(p) for p in self.params]
        self.gw1, self.gw2, self.gpre, self.glast, self.ggate = self.grads
        # the second projection's 32-blocks along hidden, the first's along 2 ffn, inside each expert
        self.s1 = torch.full((experts,), 2 * ffn, dtype=torch.int32, device=device)
        self.s2 = torch.full((experts,), hidden, dtype=torch.int32, device=device)
        self.q1 = bs.alloc_quantized(experts * 2 * ffn, hidden, experts, MX, BOTH, device)
        self.q2 = bs.alloc_quantized(experts * hidden, ffn, experts, MX, BOTH, device)
        self.quantize_weights()
        if state == "8bit":
            sizes = [p.numel() for p in self.params]
            m, v = ([torch.zeros(n, dtype=torch.uint8, device=device) for n in sizes] for _ in range(2))
            ms, vs = ([torch.zeros((n + 127) // 128, device=device) for n in sizes] for _ in range(2))
        else:
            m, v = ([torch.zeros_like(p) for p in self.params] for _ in range(2))
            ms = vs = None
        self.plan = bs.adamw_plan(self.params, self.grads, m, v, ms, vs,
                                  copies=[self.w1c, self.w2c, None, None, None], decay_scales=[1, 1, 0, 0, 0])
        self.step = 0

    def quantize_weights(self):
        bs.grouped_quantize(self.w1c, self.s1, MX, BOTH, self.q1)
        bs.grouped_quantize(self.w2c, self.s2, MX, BOTH, self.q2)

    def forward(self, x, order, splits, probs):
        """x [T, h] bf16; order: the tokens sorted by expert; splits [e]; probs [T] in that order."""
        T = x.shape[0]
        first = bs.residual_norm(x, pre_weight=self.pre, weight_offset=1.0)
        n = first["n"][order]
        xq = bs.grouped_quantize(n, splits, MX, BOTH, bs.alloc_quantized(T, self.h, self.e, MX, BOTH))
        ab = torch.empty((T, 2 * self.f), dtype=torch.bfloat16, device=self.dev)
        hq = bs.alloc_quantized(T, self.f, self.e, MX, BOTH)
        bs.grouped_gemm_swiglu(xq, self.h, self.q1, self.f, splits, T, probs=probs, ab=ab, out=hq)
        sorted_y = torch.empty((T, self.h), dtype=torch.bfloat16, device=self.dev)
        bs.grouped_gemm_fprop(hq, self.f, self.q2, self.h, splits, T, sorted_y, bs.OUT_BF16)
        y = torch.empty_like(sorted_y)
        y[order] = sorted_y
        last = bs.residual_norm(x, y, pre_weight=self.last, gate=self.gate, gate_kind=bs.GATE_CHANNEL,
                                weight_offset=1.0)
        self.kept = (x, order, splits, probs, first, xq, ab, hq, y, last)
        return last["n"]

    def backward(self, dout):
        """From dout [T, h] bf16: the parameters' gradients, and those of x and of the probabilities."""
        x, order, splits, probs, first, xq, ab, hq, y, last = self.kept
        T = x.shape[0]
        d = bs.residual_norm_grad(dout, None, last["r"], last["rstd_r"], self.last, y=y, gate=self.gate,
                                  gate_kind=bs.GATE_CHANNEL, weight_offset=1.0, dpre_weight=self.glast,
                                  dgate=self.ggate)
        dy = bs.grouped_quantize(d["dy"][order], splits, MX, BOTH, bs.alloc_quantized(T, self.h, self.e, MX, BOTH))
        dab = bs.alloc_quantized(T, 2 * self.f, self.e, MX, BOTH)
        dprobs = torch.empty(T, device=self.dev)
        bs.grouped_gemm_swiglu_grad(dy, self.h, self.q2, self.f, ab, splits, T, probs=probs, out=dab, dprobs=dprobs)
        bs.grouped_gemm_wgrad(dy, self.h, hq, self.f, splits, T, MX, self.gw2.view(self.e, self.h, self.f))
        bs.grouped_gemm_wgrad(dab, 2 * self.f, xq, self.h, splits, T, MX, self.gw1.view(self.e, 2 * self.f, self.h))
        sorted_dn = torch.empty((T, self.h), dtype=torch.bfloat16, device=self.dev)
        bs.grouped_gemm_dgrad(dab, 2 * self.f, self.q1, self.h, splits, T, sorted_dn, bs.OUT_BF16)
        dn = torch.empty_like(sorted_dn)
        dn[order] = sorted_dn
        dx = bs.residual_norm_grad(dn, d["dx"], first["r"], first["rstd_r"], self.pre, weight_offset=1.0,
                                   dpre_weight=self.gpre)["dx"]
        return dx, dprobs

    def update(self, lr, **more):
        self.step += 1
        bs.adamw_step(self.plan, lr, step=self.step, seed=self.seed, **more)  # (8-bit states: stochastic rounding)
        self.quantize_weights()


def routes(tokens, experts, generator, device="cuda"):
    """Each token's expert and probability, sorted by expert: the order, the sizes and the probabilities."""
    logits = torch.randn((tokens, experts), generator=generator, device=device)
    p, expert = torch.softmax(logits, 1).max(1)
    order = torch.argsort(expert, stable=True)
    splits = torch.bincount(expert, minlength=experts).to(torch.int32)
    return order, splits, p[order].contiguous()


def train(tokens=4096, hidden=1024, ffn=512, experts=8, steps=20, state="8bit", lr=3e-3, seed=0, log=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    teacher, layer = (ExpertLayer(hidden, ffn, experts, state, seed + 1 + i) for i in range(2))
    losses = []
    for i in range(steps):
        x = torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16()
        route = routes(tokens, experts, g)
        target = teacher.forward(x, *route).float()
        torch.cuda.synchronize()
        t = time.time()
        miss = layer.forward(x, *route).float() - target
        layer.backward((miss * (2.0 / tokens)).bfloat16())
        layer.update(lr, beta2=0.99, weight_decay=0.0)
        losses.append(miss.square().mean())
        torch.cuda.synchronize()
        if log:
            log(f"step {i + 1}: loss {float(losses[-1]):.5f}  {1e3 * (time.time() - t):.2f} ms")
    return [float(v) for v in losses]


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 4096), ("hidden", 1024), ("ffn", 512), ("experts", 8), ("steps", 20)):
        p.add_argument("--" + name, type=int, default=default)
    p.add_argument("--state", choices=["fp32", "8bit"], default="8bit")
    p.add_argument("--lr", type=float, default=3e-3)
    a = p.parse_args()
    train(a.tokens, a.hidden, a.ffn, a.experts, a.steps, a.state, a.lr, log=lambda m: print(m, flush=True))


if __name__ == "__main__":
    main()
