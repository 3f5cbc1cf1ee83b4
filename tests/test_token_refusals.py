"""What the router, the plan, the rows' movers and the 8-bit activations refuse, before any HIP call (no GPU needed): the
fake pointers are never dereferenced."""
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

P = 1 << 20
OK, NULL, GROUPS, RECIPE, SHAPE, ALIGN, LAYOUT, ARG = 0, -1, -2, -3, -4, -5, -6, -7
INF, NAN = float("inf"), float("nan")


def route(logits=P, dtype=bs.F32, tokens=4, E=8, k=2, scoring=bs.ROUTE_SOFTMAX, bias=P, renorm=1, scale=1.0, probs=P,
          experts=P, total=P, ws=P):
    return bs.lib().bsfp8_route_topk(logits, dtype, tokens, E, k, scoring, bias, renorm, scale, probs, experts, total, ws,
                                     None)


def route_grad(dprobs=P, logits=P, dtype=bs.F32, experts=P, tokens=4, E=8, k=2, scoring=bs.ROUTE_SIGMOID, renorm=0,
               scale=1.0, total=P, dlogits=P):
    return bs.lib().bsfp8_route_topk_grad(dprobs, logits, dtype, experts, tokens, E, k, scoring, renorm, scale, total,
                                          dlogits, None)


ROUTE = [(dict(E=0), GROUPS), (dict(E=1025), GROUPS), (dict(k=0), SHAPE), (dict(k=9), SHAPE), (dict(E=64, k=33), SHAPE),
         (dict(tokens=-1), SHAPE), (dict(tokens=(1 << 29) + 1), SHAPE), (dict(dtype=2), ARG), (dict(scoring=0), ARG),
         (dict(scoring=3), ARG), (dict(renorm=2), ARG), (dict(scale=INF), ARG), (dict(scale=NAN), ARG),
         (dict(logits=None), NULL), (dict(experts=None), NULL), (dict(logits=P + 8), ALIGN), (dict(experts=P + 2), ALIGN),
         (dict(total=P + 2), ALIGN)]


@pytest.mark.parametrize("change,code", ROUTE + [
    (dict(probs=None), NULL), (dict(ws=None), NULL), (dict(probs=P + 1), ALIGN), (dict(bias=P + 2), ALIGN),
    (dict(ws=P + 4), ALIGN), (dict(tokens=0, logits=None, probs=None, experts=None, total=None), OK)])
def test_route_refuses(change, code):
    assert route(**change) == code


@pytest.mark.parametrize("change,code", ROUTE + [
    (dict(dprobs=None), NULL), (dict(dlogits=None), NULL), (dict(dprobs=P + 2), ALIGN), (dict(dlogits=P + 4), ALIGN),
    (dict(tokens=0, logits=None, dprobs=None, experts=None, dlogits=None), OK)])
def test_route_gradient_refuses(change, code):
    assert route_grad(**change) == code


def plan(experts=P, probs=P, tokens=4096, k=2, E=8, splits=P, rows=P, choices=P, rprobs=P, ws=P):
    return bs.lib().bsfp8_dispatch_plan(experts, probs, tokens, k, E, splits, rows, choices, rprobs, ws, None)


@pytest.mark.parametrize("change,code", [
    (dict(E=0), GROUPS), (dict(E=1025), GROUPS), (dict(k=0), SHAPE), (dict(k=33), SHAPE), (dict(tokens=-1), SHAPE),
    (dict(tokens=(1 << 29) + 1), SHAPE), (dict(experts=None), NULL), (dict(splits=None), NULL), (dict(rows=None), NULL),
    (dict(choices=None), NULL), (dict(rprobs=None), NULL), (dict(probs=None), NULL), (dict(ws=None), NULL),
    (dict(experts=P + 2), ALIGN), (dict(splits=P + 2), ALIGN), (dict(rows=P + 1), ALIGN), (dict(choices=P + 3), ALIGN),
    (dict(rprobs=P + 2), ALIGN), (dict(ws=P + 4), ALIGN)])
def test_plan_refuses(change, code):
    assert plan(**change) == code


def move(call, x=P, dtype=bs.BF16, tokens=4, cols=64, rows=P, k=2, weights=P, out=P, cap=8, add=P, y=P, dw=P):
    L = bs.lib()
    if call == "dispatch":
        return L.bsfp8_dispatch(x, dtype, tokens, cols, rows, k, weights, out, cap, None)
    if call == "combine":
        return L.bsfp8_combine(x, dtype, cap, cols, rows, tokens, k, weights, add, out, None)
    return L.bsfp8_combine_grad(x, dtype, tokens, cols, y, cap, rows, k, weights, out, dw, None)


@pytest.mark.parametrize("call", ["dispatch", "combine", "grad"])
@pytest.mark.parametrize("change,code", [
    (dict(tokens=-1), SHAPE), (dict(cols=0), SHAPE), (dict(cols=(1 << 24) + 1), SHAPE), (dict(k=0), SHAPE),
    (dict(k=33), SHAPE), (dict(cap=-1), SHAPE), (dict(cap=1 << 31), SHAPE), (dict(dtype=5), ARG), (dict(x=None), NULL),
    (dict(rows=None), NULL), (dict(x=P + 8), ALIGN), (dict(rows=P + 2), ALIGN), (dict(weights=P + 2), ALIGN),
    (dict(out=P + 8), ALIGN), (dict(tokens=0, x=None, rows=None, out=None, dw=None), OK)])
def test_movers_refuse(call, change, code):
    assert move(call, **change) == code


def test_movers_refuse_more():
    assert move("dispatch", out=None) == NULL and move("combine", out=None) == NULL
    assert move("dispatch", cap=0, out=None) == OK
    assert move("combine", add=P + 4) == ALIGN
    assert move("grad", out=None, dw=None) == ARG and move("grad", y=None) == NULL
    assert move("grad", y=P + 8) == ALIGN and move("grad", dw=P + 2) == ALIGN


def quantize(x=P, tokens=4, cols=64, choices=P, k=2, weights=P, cap=8, splits=P, E=2, recipe=bs.RECIPE_MX, which=3, rq=P,
             rs=P, cq=P, cs=P, status=P):
    return bs.lib().bsfp8_dispatch_quantize(x, tokens, cols, choices, k, weights, cap, splits, E, recipe, which, rq, rs, cq,
                                            cs, status, None)


LAYOUTS = [(dict(recipe=9), RECIPE), (dict(recipe=bs.RECIPE_PC), LAYOUT), (dict(recipe=bs.RECIPE_MX | bs.GEMM_FP8_MFMA), RECIPE),
           (dict(which=4), ARG), (dict(cols=48), SHAPE), (dict(cols=0), SHAPE), (dict(cap=-1), SHAPE), (dict(cap=(1 << 24) - 254), SHAPE),
           (dict(E=0), GROUPS), (dict(E=1025), GROUPS), (dict(splits=None), NULL), (dict(rq=None), NULL), (dict(rs=None), NULL),
           (dict(cq=None), NULL), (dict(cs=None), NULL), (dict(rq=P + 8), ALIGN), (dict(cs=P + 8), ALIGN),
           (dict(splits=P + 2), ALIGN), (dict(status=P + 1), ALIGN)]


@pytest.mark.parametrize("change,code", LAYOUTS + [
    (dict(which=0), ARG), (dict(x=None), NULL), (dict(choices=None), NULL), (dict(x=P + 8), ALIGN),
    (dict(choices=P + 2), ALIGN), (dict(weights=P + 2), ALIGN), (dict(k=40), SHAPE),
    (dict(cap=0, x=None, choices=None, splits=None, rq=None), OK)])
def test_dispatch_quantize_refuses(change, code):
    assert quantize(**change) == code


def keep(act=bs.ACT_SWIGLU, h=P, probs=P, cap=8, cols=64, splits=P, E=2, recipe=bs.RECIPE_MX, which=3, rq=P, rs=P, cq=P,
         cs=P, kq=P, ks=P, status=P):
    return bs.lib().bsfp8_grouped_act_checkpoint(act, h, probs, cap, cols, splits, E, recipe, which, rq, rs, cq, cs, kq, ks,
                                                 status, None)


def keep_grad(act=bs.ACT_SRELU, kq=P, ks=P, probs=P, dy=P, cap=8, cols=64, splits=P, E=2, recipe=bs.RECIPE_MX, which=3,
              rq=P, rs=P, cq=P, cs=P, yq=P, ys=P, dp=P, ws=P, status=P):
    return bs.lib().bsfp8_grouped_act_checkpoint_grad(act, kq, ks, probs, dy, cap, cols, splits, E, recipe, which, rq, rs,
                                                      cq, cs, yq, ys, dp, ws, status, None)


KEEP = LAYOUTS + [(dict(act=0), ARG), (dict(act=bs.ACT_SRELU_GRAD), ARG), (dict(act=bs.ACT_SWIGLU_GRAD), ARG),
                  (dict(cols=(1 << 21) + 32), SHAPE), (dict(kq=None), NULL),
                  (dict(ks=None), NULL), (dict(kq=P + 4), ALIGN), (dict(ks=P + 4), ALIGN), (dict(probs=P + 2), ALIGN),
                  (dict(cap=0, kq=None, rq=None), OK)]


@pytest.mark.parametrize("change,code", KEEP + [(dict(which=0), ARG), (dict(h=None), NULL), (dict(h=P + 8), ALIGN)])
def test_checkpoint_refuses(change, code):
    assert keep(**change) == code


@pytest.mark.parametrize("change,code", KEEP + [
    (dict(which=0, yq=None, ys=None, dp=None), ARG), (dict(dy=None), NULL), (dict(yq=None), NULL), (dict(ys=None), NULL),
    (dict(ws=None), NULL), (dict(dy=P + 8), ALIGN), (dict(yq=P + 8), ALIGN), (dict(dp=P + 2), ALIGN),
    (dict(ws=P + 8), ALIGN)])
def test_checkpoint_gradient_refuses(change, code):
    assert keep_grad(**change) == code


def test_workspace_bytes():
    assert bs.route_topk_workspace_bytes(-1, 8) == 0 and bs.route_topk_workspace_bytes(5, 0) == 0
    assert bs.route_topk_workspace_bytes(0, 8) == 0 and bs.route_topk_workspace_bytes(1 << 20, 128) % (4 * 128) == 0
    assert bs.dispatch_plan_workspace_bytes(4096, 1, 8) == 0  # one launch
    assert bs.dispatch_plan_workspace_bytes(4097, 1, 8) >= 2 * 9 * 4
    assert bs.dispatch_plan_workspace_bytes(1 << 25, 32, 1024) <= 512 * 1028 * 4
    assert bs.grouped_act_checkpoint_grad_workspace_bytes(100, 160) >= 100 * 4
    assert bs.grouped_act_checkpoint_grad_workspace_bytes(100, 40) == 0


def test_binding_checks():
    """Host memory, wrong types and wrong shapes are refused before the library is called."""
    l, e = torch.zeros(4, 8), torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="device memory"):
        bs.route_topk(l, 2, stream=0)
    with pytest.raises(TypeError, match="logits"):
        bs.route_topk(l.double(), 2, stream=0)
    with pytest.raises(ValueError, match="two-dimensional"):
        bs.route_topk(l[0], 2, stream=0)
    with pytest.raises(ValueError, match="two-dimensional"):
        bs.dispatch_plan(None, 2, stream=0)
    with pytest.raises(TypeError, match="experts"):
        bs.dispatch_plan(e.long(), 2, stream=0)
    with pytest.raises(ValueError, match="device memory"):
        bs.dispatch(l, {"rows": e}, stream=0)
    with pytest.raises(TypeError, match="h: dtype"):
        bs.grouped_act_checkpoint(bs.ACT_SRELU, l, e[0], bs.RECIPE_MX, 1, {}, {}, stream=0)
