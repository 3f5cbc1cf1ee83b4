"""The example's expert layer: its gradients against autograd through the same formulas in 64 bits, on the
values that its quantized operands stand for, and a few steps that fit."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import block_scaled_fp8_grouped_amd as bs
import expert_layer

pytestmark = pytest.mark.gpu


def reference(layer, x, order, splits, probs, dr):
    """The layer by torch in 64 bits from its master weights, and the gradients of sum(r dr)."""
    names = ("w1", "w2", "pre", "last", "gate")
    v = {k: getattr(layer, k).double().requires_grad_() for k in names}
    x = x.double().requires_grad_()
    p = probs.double().requires_grad_()

    def norm(t, w):
        return t * (t.square().mean(1, keepdim=True) + 1e-6).rsqrt() * (w + 1)

    n = norm(x, v["pre"])[order]
    w1, w2 = v["w1"].view(layer.e, 2 * layer.f, layer.h), v["w2"].view(layer.e, layer.h, layer.f)
    parts, at = [], 0
    for e, k in enumerate(splits.tolist()):
        a, b = (n[at:at + k] @ w1[e].t()).chunk(2, 1)
        parts.append((torch.nn.functional.silu(a) * b * p[at:at + k, None]) @ w2[e].t())
        at += k
    y = torch.empty_like(x)
    y = y.index_copy(0, order, torch.cat(parts))
    r = norm(x + v["gate"] * y, v["last"])
    (r * dr.double()).sum().backward()
    return r.detach(), {k: t.grad for k, t in v.items()}, x.grad, p.grad


@pytest.mark.parametrize("tokens,hidden,ffn,experts", [(40, 96, 64, 5), (700, 160, 96, 7)])
def test_gradients(tokens, hidden, ffn, experts):
    """Every operand is rounded to e4m3 on the way (each value off by up to 2^-4, the rms of a uniform
    rounding error 2^-4 / sqrt(3) of it): a sum of such products is off by that share of its norm for each of
    its at most five rounded factors in a row, 0.036 sqrt(5) < 0.1; twice that is allowed."""
    g = torch.Generator(device="cuda").manual_seed(1)
    layer = expert_layer.ExpertLayer(hidden, ffn, experts, "fp32", 3)
    x = torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16()
    route = expert_layer.routes(tokens, experts, g)
    dr = torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16()
    r = layer.forward(x, *route)
    dx, dprobs = layer.backward(dr)
    rr, grads, rx, rp = reference(layer, x, *route, dr)

    def off(a, b):
        return float((a.double() - b).norm() / b.norm())

    assert off(r, rr) < 0.2 and off(dx, rx) < 0.2 and off(dprobs, rp) < 0.2
    for k, got in zip(("w1", "w2", "pre", "last", "gate"), layer.grads):
        assert off(got, grads[k]) < 0.2, k


@pytest.mark.parametrize("state", ["fp32", "8bit"])
def test_a_few_steps_fit(state):
    losses = expert_layer.train(tokens=1024, hidden=256, ffn=128, experts=4, steps=30, state=state)
    assert losses[-1] < 0.7 * losses[0]
