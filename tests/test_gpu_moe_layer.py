"""The example's mixture-of-experts layer: its output and gradients against autograd through the same formulas in 64
bits, with the experts that the layer chose, and that it runs."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer

pytestmark = pytest.mark.gpu


def reference(layer, x, experts, dr):
    """The layer by torch in 64 bits from its master weights, and the gradients of sum(r dr) + balance * its loss."""
    names = ("router", "w1", "w2", "pre", "last", "gate")
    v = {k: getattr(layer, k).double().requires_grad_() for k in names}
    x = x.double().requires_grad_()
    T, experts = x.shape[0], experts.long()

    def norm(t, w):
        return t * (t.square().mean(1, keepdim=True) + 1e-6).rsqrt() * (w + 1)

    n = norm(x, v["pre"])
    scores = torch.softmax(n @ v["router"].t(), 1)
    p = scores.gather(1, experts)
    p = p / p.sum(1, keepdim=True)
    p.retain_grad()
    w1, w2 = v["w1"].view(layer.e, 2 * layer.f, layer.h), v["w2"].view(layer.e, layer.h, layer.f)
    y = torch.zeros_like(x)
    for e in range(layer.e):
        t, j = (experts == e).nonzero(as_tuple=True)
        a, b = (n[t] @ w1[e].t()).chunk(2, 1)
        y = y.index_add(0, t, (torch.nn.functional.silu(a) * b * p[t, j, None]) @ w2[e].t())
    r = norm(x + v["gate"] * y, v["last"])
    share = torch.bincount(experts.flatten(), minlength=layer.e).double() / experts.numel()
    balance = layer.e * (share * scores.mean(0)).sum()
    ((r * dr.double()).sum() + layer.balance * balance).backward()
    # the chosen logits' gradients before their differences, and what they make of the router's, token by token
    size = p * (p.grad.abs() + (p * p.grad.abs()).sum(1, keepdim=True))
    size = float((size.norm(dim=1) * n.norm(dim=1)).norm().detach())
    return r.detach(), float(balance.detach()), {k: t.grad for k, t in v.items()}, x.grad, size


@pytest.mark.parametrize("keep", ["bf16", "8bit"])
@pytest.mark.parametrize("tokens,hidden,ffn,experts,k", [(1, 96, 64, 5, 2), (40, 96, 64, 5, 1), (300, 160, 96, 7, 3),
                                                         (9, 64, 32, 40, 6)])
def test_gradients(tokens, hidden, ffn, experts, k, keep):
    """Operands are rounded to e4m3 on the way (each value off by up to 2^-4, the rms of a uniform rounding error
    2^-4 / sqrt(3) of it): a sum of such products is off by that share of its norm for each of its rounded factors in a
    row, at most seven with the activation's input kept in 8 bits, 0.036 sqrt(7) < 0.1; twice that is allowed.  The
    router's gradient is made of differences of such sums within a token, which may cancel: there the share is one of
    the sums before the difference."""
    g = torch.Generator(device="cuda").manual_seed(1)
    layer = moe_layer.MoELayer(hidden, ffn, experts, k, keep, balance=1.0, seed=3)
    x = torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16()
    dr = torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16()
    r = layer.forward(x)
    dx = layer.backward(dr)
    chosen = layer.kept[3]["experts"]
    assert bool(((chosen >= 0) & (chosen < experts)).all())
    rr, balance, grads, rx, size = reference(layer, x, chosen, dr)

    def off(a, b):
        return float((a.double() - b).norm() / b.norm())

    assert off(r, rr) < 0.2 and off(dx, rx) < 0.2
    assert abs(float(layer.balance_loss) - balance) < 0.01 * balance  # (n rounded to bf16, 2^-8 of each of the logits' terms)
    for name, got in zip(("w1", "w2", "pre", "last", "gate"), layer.grads[1:]):
        assert off(got, grads[name]) < 0.2, name
    assert float((layer.grads[0].double() - grads["router"]).norm()) < 0.2 * (size + float(grads["router"].norm()))


def test_both_ways_of_keeping_agree():
    """The same layer kept in bf16 and in 8 bits: each within 0.1 (half of what is allowed above) of the formulas' norm."""
    layers = [moe_layer.MoELayer(128, 96, 6, 2, keep, seed=5) for keep in ("bf16", "8bit")]
    g = torch.Generator(device="cuda").manual_seed(2)
    x, dr = (torch.randn((500, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    outs = [(l.forward(x), l.backward(dr)) for l in layers]
    assert torch.equal(layers[0].kept[3]["experts"], layers[1].kept[3]["experts"])
    for a, b in [*zip(*outs), *zip(layers[0].grads, layers[1].grads)]:
        assert float((a.double() - b.double()).norm()) < 0.2 * float(a.double().norm())


@pytest.mark.parametrize("keep", ["bf16", "8bit"])
def test_runs(keep):
    losses = moe_layer.train(tokens=200, hidden=128, ffn=64, experts=8, top_k=2, steps=3, keep=keep)
    assert len(losses) == 3 and all(v == v and v < 100 for v in losses)
