"""The calls for routing, tokens and kept activations by every way they can be made: a run of them together, the native
host path and the ctypes path, given streams, two streams at once, captured graphs, arrays of more than 2^31 elements.
Every way gives the same bits."""
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
MX, ROW, COL, BOTH = bs.RECIPE_MX, bs.ROWWISE, bs.COLWISE, bs.ROWWISE | bs.COLWISE


class Run:
    """One layer's calls in order on given tensors (all outputs and workspaces allocated here, or by each call)."""

    def __init__(self, tokens=300, experts=12, k=3, cols=160, seed=0, act=bs.ACT_SWIGLU, given=True):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.T, self.E, self.k, self.c, self.R, self.act, self.given = tokens, experts, k, cols, tokens * k, act, given
        self.wide = cols * (2 if act == bs.ACT_SWIGLU else 1)
        rand = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
        self.logits, self.dsum, self.bias = rand(tokens, experts), rand(experts), rand(experts)
        self.x, self.h, self.dy = rand(tokens, cols).to(BF16), rand(self.R, self.wide).to(BF16), rand(self.R, cols).to(BF16)
        if given:
            self.alloc()

    def alloc(self):
        new = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device=DEV)  # noqa: E731
        T, k, E, R, c = self.T, self.k, self.E, self.R, self.c
        i32 = torch.int32
        self.o = dict(probs=new(T, k), experts=new(T, k, dtype=i32), score_sum=new(E),
                      route_ws=new(max(1, bs.route_topk_workspace_bytes(T, E)), dtype=torch.uint8),
                      plan=dict(splits=new(E, dtype=i32), rows=new(T, k, dtype=i32), choices=new(R, dtype=i32),
                                probs=new(R)),
                      plan_ws=new(max(1, bs.dispatch_plan_workspace_bytes(T, k, E)), dtype=torch.uint8),
                      rows=new(R, c, dtype=BF16), out=new(T, c, dtype=BF16), dy=new(R, c, dtype=BF16), dweights=new(T, k),
                      dlogits=new(T, E), dprobs=new(R), status=new(1, dtype=i32),
                      grad_ws=new(max(1, bs.grouped_act_checkpoint_grad_workspace_bytes(R, c)), dtype=torch.uint8))
        self.q = self.layouts()

    def layouts(self):
        q = lambda cols, which: {n: t.zero_() for n, t in  # noqa: E731 (rows behind the last are compared too)
                                 bs.alloc_quantized(self.R, cols, self.E, MX, which, DEV).items()}
        return dict(x=q(self.c, BOTH), a=q(self.c, BOTH), kept=q(self.wide, ROW), g=q(self.wide, BOTH), y=q(self.c, COL))

    def __call__(self, stream=None):
        kw = dict(stream=stream)
        o = self.o if self.given else None
        pick = (lambda **names: {a: o[n] for a, n in names.items()}) if self.given else (lambda **names: {})
        q = self.q if self.given else self.layouts()
        route = bs.route_topk(self.logits, self.k, bs.ROUTE_SIGMOID, self.bias, scale=2.5, **kw, **(
            pick(probs="probs", experts="experts", score_sum="score_sum", workspace="route_ws") if self.given else
            dict(score_sum=torch.empty(self.E, device=DEV))))
        plan = bs.dispatch_plan(route["experts"], self.E, route["probs"], **kw, **pick(out="plan", workspace="plan_ws"))
        w = route["probs"]
        zeros = {} if self.given else dict(out=torch.zeros((self.R, self.c), dtype=BF16, device=DEV))
        rows = bs.dispatch(self.x, plan, weights=w, **kw, **(pick(out="rows") or zeros))
        bs.dispatch_quantize(self.x, plan, MX, BOTH, q["x"], **kw, **pick(status="status"))
        bs.grouped_act_checkpoint(self.act, self.h, plan["splits"], MX, BOTH, q["a"], q["kept"], probs=plan["probs"], **kw)
        dprobs = o["dprobs"] if self.given else torch.zeros(self.R, device=DEV)
        bs.grouped_act_checkpoint_grad(self.act, q["kept"], self.dy, plan["splits"], MX, BOTH, q["g"],
                                       probs=plan["probs"], y=q["y"], dprobs=dprobs, **kw, **pick(workspace="grad_ws"))
        out = bs.combine(rows, plan, weights=w, add=self.x, **kw, **pick(out="out"))
        d = bs.combine_grad(out, plan, y=rows, weights=w, **kw, **(pick(dy="dy", dweights="dweights") or dict(
            dy=torch.zeros((self.R, self.c), dtype=BF16, device=DEV))))
        dlogits = bs.route_topk_grad(d["dweights"], self.logits, route["experts"], bs.ROUTE_SIGMOID, True, 2.5,
                                     dscore_sum=self.dsum, **kw, **pick(dlogits="dlogits"))
        got = dict(route, rows=rows, out=out, dy=d["dy"], dweights=d["dweights"], dlogits=dlogits, dprobs=dprobs)
        got.update({f"plan {n}": t for n, t in plan.items()})
        got.update({f"{a} {n}": t for a, l in q.items() for n, t in l.items()})
        return got


def copied(got):
    torch.cuda.synchronize()
    return {n: t.clone() for n, t in got.items()}


def same(a, b):
    assert set(a) == set(b)
    for n in a:
        assert a[n].dtype == b[n].dtype and torch.equal(a[n].flatten().view(torch.uint8), b[n].flatten().view(torch.uint8)), n


SIZES = [dict(tokens=1, experts=8, k=2, cols=64), dict(), dict(tokens=2500, experts=130, k=5, cols=416),
         dict(tokens=77, experts=1, k=1, cols=32, act=bs.ACT_SRELU)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("given", [True, False])
def test_native_and_ctypes_paths_agree(monkeypatch, size, given):
    native = copied(Run(**size, given=given)())
    assert bool(native["out"].isfinite().all()) and bool((native["experts"] >= 0).all())
    with monkeypatch.context() as m:
        m.setattr(bs, "_native", None)
        same(copied(Run(**size, given=given)()), native)


@pytest.mark.parametrize("native", [True, False])
def test_both_paths_refuse_alike(monkeypatch, native):
    if not native:
        monkeypatch.setattr(bs, "_native", None)
    r = Run()
    plan = bs.dispatch_plan(torch.zeros((r.T, r.k), dtype=torch.int32, device=DEV), r.E)
    x, half = r.x, r.x[:, ::2]
    q = r.q["x"]
    for error, call in (
            (bs.BSFP8Error, lambda: bs.route_topk(r.logits, 13)), (bs.BSFP8Error, lambda: bs.route_topk(r.logits, 0)),
            (bs.BSFP8Error, lambda: bs.route_topk(r.logits, 2, scoring=7)),
            (TypeError, lambda: bs.route_topk(r.logits.double(), 2)), (ValueError, lambda: bs.route_topk(r.logits.t(), 2)),
            (ValueError, lambda: bs.route_topk(r.logits, 2, bias=r.bias[:5])),
            (ValueError, lambda: bs.route_topk(r.logits, 2, probs=torch.empty((r.T, 3), device=DEV))),
            (ValueError, lambda: bs.route_topk(r.logits.cpu(), 2)),
            (ValueError, lambda: bs.route_topk_grad(r.o["dweights"][:5], r.logits, r.o["experts"], 0, True, 1.0)),
            (TypeError, lambda: bs.route_topk_grad(r.o["dweights"], r.logits, r.o["dweights"], 0, True, 1.0)),
            (TypeError, lambda: bs.dispatch_plan(r.o["probs"], 4)),
            (ValueError, lambda: bs.dispatch_plan(r.o["experts"], 4, probs=r.o["probs"][:2])),
            (ValueError, lambda: bs.dispatch(half, plan)), (TypeError, lambda: bs.dispatch(x.half(), plan)),
            (ValueError, lambda: bs.dispatch(x[:9], plan)), (ValueError, lambda: bs.dispatch(x, plan, out=r.o["rows"][:, :8])),
            (ValueError, lambda: bs.dispatch(x, plan, weights=r.o["probs"].t())),
            (TypeError, lambda: bs.dispatch_quantize(x.float(), plan, MX, BOTH, q)),
            (ValueError, lambda: bs.dispatch_quantize(x[:9], plan, MX, BOTH, q)),
            (TypeError, lambda: bs.combine(r.dy, plan, add=x.float())), (ValueError, lambda: bs.combine(r.dy, plan, add=x[:9])),
            (ValueError, lambda: bs.combine(r.dy, plan, out=x[:9])),
            (ValueError, lambda: bs.combine_grad(x, plan, y=r.dy[:, :8])),
            (TypeError, lambda: bs.combine_grad(x, plan, y=r.dy.float())),
            (TypeError, lambda: bs.grouped_act_checkpoint(r.act, r.h.float(), plan["splits"], MX, BOTH, r.q["a"], r.q["kept"])),
            (ValueError, lambda: bs.grouped_act_checkpoint(r.act, r.h, plan["splits"], MX, BOTH, r.q["a"], r.q["kept"],
                                                           probs=r.o["dprobs"][:7])),
            (ValueError, lambda: bs.grouped_act_checkpoint_grad(r.act, r.q["kept"], r.dy[:, :32], plan["splits"], MX, BOTH,
                                                                r.q["g"]))):
        with pytest.raises(error):
            call()
    torch.cuda.synchronize()
    assert not any(bool(t.any()) for t in q.values()) and not bool(r.o["rows"].any())


def test_given_streams():
    want = copied(Run()())
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0, torch.cuda.default_stream()):
        for given in (True, False):
            r = Run(given=given)
            torch.cuda.synchronize()
            got = r(stream)
            torch.cuda.synchronize()
            same(copied(got), want)


def test_two_streams_at_once():
    runs = [Run(2500, 130, 5, 416, seed=s) for s in (1, 2)]
    want = [copied(r()) for r in runs]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [r(s) for r, s in zip(runs, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        same(copied(a), b)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("given", [True, False])
def test_captured_and_replayed(size, given):
    r = Run(**size, given=given)
    copied(r())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = r()
    for seed in range(4):
        other = Run(**size, seed=seed + 10, given=given)
        want = copied(other())  # (eager work between the replays)
        for name in ("logits", "x", "h", "dy", "dsum", "bias"):
            getattr(r, name).copy_(getattr(other, name))
        for t in got.values():  # (what lies behind a layout's last group is left as it was, and the groups' sizes change)
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        same(copied(got), want)


def test_two_graphs_of_one_layer_share_nothing_they_should_not():
    """Two captured graphs with workspaces of their own replayed at once on two streams."""
    runs = [Run(2500, 130, 5, 416, seed=s) for s in (3, 4)]
    want = [copied(r()) for r in runs]
    graphs, got = [], []
    for r in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(r())
        graphs.append(g)
    for _ in range(3):
        streams = [torch.cuda.Stream() for _ in runs]
        for g, s in zip(graphs, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            same(copied(a), b)


# --------------------------------------------------------------- arrays of more than 2^31 elements

def tail_of(rows, cols, tail, dtype=BF16):
    """[rows][cols] zeros with random values in the last rows, and those alone."""
    t = torch.zeros((rows, cols), dtype=dtype, device=DEV)
    t[-tail:] = torch.randn((tail, cols), device=DEV).to(dtype)
    return t, t[-tail:].clone()


@pytest.mark.parametrize("scoring", [bs.ROUTE_SOFTMAX, bs.ROUTE_SIGMOID])
def test_large_router(scoring):
    experts, tail, k = 1024, 37, 8
    l, small = tail_of((1 << 31) // experts + 50, experts, tail)
    big, one = bs.route_topk(l, k, scoring), bs.route_topk(small, k, scoring)
    for n in one:
        assert torch.equal(big[n][-tail:], one[n]), n
    dp = torch.randn_like(big["probs"])
    s = torch.randn(experts, device=DEV)
    d = bs.route_topk_grad(dp, l, big["experts"], scoring, True, 1.0, dscore_sum=s)
    e = bs.route_topk_grad(dp[-tail:].clone(), small, one["experts"], scoring, True, 1.0, dscore_sum=s)
    assert torch.equal(d[-tail:], e) and bool(e.any())


def test_large_dispatch():
    """Rows past 2^31 elements, by tokens that lie past it as well: the last tokens at the second expert."""
    cols, tail = 8192, 200
    tokens = (1 << 31) // cols + 300
    x, small = tail_of(tokens, cols, tail)
    e = torch.zeros((tokens, 1), dtype=torch.int32, device=DEV)
    e[-tail:] = 1
    w = torch.rand((tokens, 1), device=DEV)
    plan = bs.dispatch_plan(e, 2)
    part = bs.dispatch_plan(e[-tail:].clone(), 2)
    rows, want = bs.dispatch(x, plan, w), bs.dispatch(small, part, w[-tail:].clone())
    assert torch.equal(rows[-tail:], want) and bool(want.any())
    assert torch.equal(bs.combine(rows, plan, w, add=x)[-tail:], bs.combine(want, part, w[-tail:].clone(), add=small))
    a = bs.combine_grad(x, plan, rows, w, dy=rows)  # (dy over y)
    b = bs.combine_grad(small, part, None, w[-tail:].clone())
    assert torch.equal(a["dy"][-tail:], b["dy"])
    # (a sum of cols products: chains of at most cols / 64 a lane, 6 steps and 8 waves)
    terms = small.double() * want.double()
    off = (a["dweights"][-tail:, 0].double() - terms.sum(1)).abs()
    assert (off <= (cols / 64 + 16) * 2.0 ** -24 * terms.abs().sum(1)).all() and bool(a["dweights"][-tail:].any())
    del rows, a
    q = bs.dispatch_quantize(x, plan, MX, BOTH, bs.alloc_quantized(tokens, cols, 2, MX, BOTH))
    p = bs.dispatch_quantize(small, part, MX, BOTH, bs.alloc_quantized(tail, cols, 2, MX, BOTH))
    assert torch.equal(q["row_q"][-tail:], p["row_q"]) and torch.equal(q["row_s"][:, -tail:], p["row_s"])
    at = (tokens - tail + 127) // 128 * 128  # the first expert's rows, in whole 128s
    n = (tail + 127) // 128 * 128
    assert torch.equal(q["col_q"][at * cols:(at + n) * cols], p["col_q"][:n * cols])
    assert torch.equal(q["col_s"][at * cols // 32:(at + n) * cols // 32], p["col_s"][:n * cols // 32])


@pytest.mark.parametrize("act", [bs.ACT_SRELU, bs.ACT_SWIGLU])
def test_large_checkpoint(act):
    cols, tail = 8192, 200
    wide = cols * (2 if act == bs.ACT_SWIGLU else 1)
    rows = (1 << 31) // cols + 300
    h, hs = tail_of(rows, wide, tail)
    dy, ds = tail_of(rows, cols, tail)
    splits = torch.tensor([rows - tail, tail], dtype=torch.int32, device=DEV)
    one = torch.tensor([0, tail], dtype=torch.int32, device=DEV)
    at, n = (rows - tail + 127) // 128 * 128, (tail + 127) // 128 * 128

    def run(h, dy, splits):
        R = h.shape[0]
        q, kept = bs.alloc_quantized(R, cols, 2, MX, BOTH), bs.alloc_quantized(R, wide, 2, MX, ROW)
        bs.grouped_act_checkpoint(act, h, splits, MX, BOTH, q, kept)
        out = {f"a {k}": v for k, v in q.items()}
        g, y, dp = bs.alloc_quantized(R, wide, 2, MX, BOTH), bs.alloc_quantized(R, cols, 2, MX, COL), torch.empty(R, device=DEV)
        bs.grouped_act_checkpoint_grad(act, kept, dy, splits, MX, BOTH, g, y=y, dprobs=dp)
        out.update({f"kept {k}": v for k, v in kept.items()})
        out.update({f"g {k}": v for k, v in g.items()})
        out.update({f"y {k}": v for k, v in y.items()})
        return out, dp

    (big, bp), (small, sp) = run(h, dy, splits), run(hs, ds, one)
    # a sum's order goes by the number of rows: both are within cols steps of what the terms add up to, which are at most
    # |dy| h^2 or |dy a b| (|silu(a)| <= |a|) with the values kept off by 2^-4 each
    v = hs.double().abs()
    size = (ds.double().abs() * (v[:, :cols] * v[:, -cols:])).sum(1) * (1 + 2.0 ** -4) ** 2
    assert ((bp[-tail:] - sp).double().abs() <= 2 * cols * 2.0 ** -24 * size).all() and bool(sp.any())
    for name, want in small.items():
        got, per = big[name], 32 if name.endswith("_s") else 1
        c = wide if name[0] in "kg" else cols
        if "row_q" in name:
            assert torch.equal(got[-tail:], want), name
        elif "row_s" in name:
            assert torch.equal(got[:, -tail:], want), name
        else:
            assert torch.equal(got[at * c // per:(at + n) * c // per], want[:n * c // per]), name


def test_more_tokens_than_a_launch_has_waves():
    """Rows of one channel: each token's part of the gradient by itself."""
    tokens = (1 << 26) + 5
    rows = torch.arange(tokens - 1, -1, -1, dtype=torch.int32, device=DEV).view(tokens, 1)
    x, y, w = (torch.rand((tokens, 1), device=DEV) for _ in range(3))
    d = bs.combine_grad(x, {"rows": rows}, y=y, weights=w)
    assert torch.equal(d["dweights"], x * y.flip(0)) and torch.equal(d["dy"], (x * w).flip(0))
    assert torch.equal(bs.combine(y, {"rows": rows}, w), y.flip(0) * w)
    assert torch.equal(bs.dispatch(x, {"rows": rows}), x.flip(0))


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("cols", [1, 8, 513, 576, 577, 1025, 1152, 1153, 2050, 2305, 4097, 8200])
@pytest.mark.parametrize("tokens,k", [(3, 1), (65, 5)])
def test_gradient_of_sums_at_every_width(dtype, cols, tokens, k):
    """Rows of one wave, of several and of several passes.  A product is rounded once (half a step); a weight's gradient is a
    chain of at most 8 ceil(cols / 512) products a lane, 6 steps and 8 waves in fp32."""
    g = torch.Generator(device=DEV).manual_seed(cols)
    rand = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    rows = torch.randperm(tokens * k, generator=g, device=DEV).to(torch.int32).view(tokens, k)
    rows[0, 0] = -1
    x, y, w = rand(tokens, cols).to(dtype), rand(tokens * k, cols).to(dtype), rand(tokens, k)
    dy = torch.full_like(y, 7.0)
    d = bs.combine_grad(x, {"rows": rows}, y=y, weights=w, dy=dy)
    live = rows >= 0
    at = rows[live].long()
    want = (x.double()[:, None] * w.double()[..., None])[live]
    assert ((dy[at].double() - want).abs() <= (torch.finfo(dtype).eps / 2 + 2.0 ** -24) * want.abs()).all()
    left = torch.ones(tokens * k, dtype=torch.bool, device=DEV)
    left[at] = False
    assert int(left.sum()) == 1 and bool((dy[left] == 7).all())
    terms = (x.double()[:, None] * torch.ones_like(w.double())[..., None])[live] * y[at].double()
    bound = (8 * ((cols + 511) // 512) + 14) * 2.0 ** -24 * terms.abs().sum(1)
    assert ((d["dweights"][live].double() - terms.sum(1)).abs() <= bound).all() and float(d["dweights"][0, 0]) == 0
    assert torch.equal(bs.combine_grad(x, {"rows": rows}, y=y, weights=w, dy=False)["dweights"], d["dweights"])
    again = bs.combine_grad(x, {"rows": rows}, y=y, weights=w, dy=y)  # (dy over y)
    assert torch.equal(again["dweights"], d["dweights"]) and torch.equal(y[at], dy[at])
