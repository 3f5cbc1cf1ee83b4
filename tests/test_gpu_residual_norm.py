"""Residual norms and their gradient against their formulas in 64 bits.

Tolerances.  An output is rounded once: half a step h of its type (bf16 2^-8, fp32 2^-24) times its
value.  Before that every number comes from a few fp32 operations on terms of a known size, with
statistics that are sums of `cols` terms taken as chains of at most 8 * 4 per thread, 6 lane steps
and 16 waves, so their relative error is at most 64 * 2^-24 = 2^-18; the sum of the sizes of an
output's terms times 2^-17 covers both.  A sum over rows is a chain of at most
rows / slots + slots / 16 + 20 terms."""
import pytest
import torch

import block_scaled_fp8_grouped_amd as bs

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
GATES = {"none": bs.GATE_NONE, "channel": bs.GATE_CHANNEL, "token": bs.GATE_TOKEN}


def close(got, ref, mag, more=2.0 ** -17):
    err = (got.double() - ref).abs()
    tol = HALF[got.dtype] * ref.abs() + more * mag + 1e-30
    bad = ~(err <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float((err / tol).max()):.3g} times the bound"


def case(rows, cols, stream, gate, seed=0, big=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rand(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device=DEV) * scale

    s = dict(x=(rand(rows, cols) * 2 * big).to(stream), y=(rand(rows, cols, scale=3.0) * big).bfloat16(),
             post=rand(cols, scale=0.3), pre=rand(cols, scale=0.3), dn=rand(rows, cols).bfloat16(),
             dr=rand(rows, cols).to(stream))
    s["gate"] = None if gate == "none" else torch.sigmoid(rand(cols if gate == "channel" else rows))
    s["kind"] = GATES[gate]
    return s


def gate64(s):
    if s["gate"] is None:
        return torch.ones((), dtype=torch.float64, device=DEV)
    g = s["gate"].double()
    return g[:, None] if s["kind"] == bs.GATE_TOKEN else g


def forward64(s, xs=1.0, ys=1.0, eps=1e-6, off=0.0, x=None, y=None, post=None, pre=None, gate=None):
    """(r, n, rstd_y, rstd_r, size of r's terms) in 64 bits."""
    x = s["x"].double() if x is None else x
    y = s["y"].double() if y is None else y
    ry = (y.square().mean(1, keepdim=True) + eps).rsqrt()
    z = y * ry * ((s["post"].double() if post is None else post) + off)
    b = ys * (gate64(s) if gate is None else gate) * z
    r = xs * x + b
    rr = (r.square().mean(1, keepdim=True) + eps).rsqrt()
    w = (s["pre"].double() if pre is None else pre) + off
    return r, r * rr * w, ry[:, 0], rr[:, 0], (xs * x).abs() + b.abs(), w


SHAPES = [(1, 1), (3, 7), (5, 8), (2, 511), (4, 513), (9, 1000), (3, 2048), (4, 2050), (3, 4097), (2, 7168), (3, 8191),
          (2, 8193), (1, 16385), (2, 32768)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("stream,gate", [(torch.bfloat16, "channel"), (torch.float32, "token"),
                                         (torch.float32, "none")])
def test_forward(rows, cols, stream, gate):
    s = case(rows, cols, stream, gate)
    kw = dict(x_scale=0.75, y_scale=-1.5, weight_offset=1.0, eps=1e-5)
    out = bs.residual_norm(s["x"], s["y"], s["post"], s["pre"], s["gate"], s["kind"], **kw)
    r, n, ry, rr, mag, w = forward64(s, 0.75, -1.5, 1e-5, 1.0)
    close(out["r"], r, mag)
    close(out["n"], n, mag * rr[:, None] * w.abs() + n.abs())
    close(out["rstd_y"], ry, ry)
    # rstd_r's sum is of squares of r, each with r's own error: twice the relative size of r's terms
    close(out["rstd_r"], rr, rr * (1 + 2 * (mag.square().mean(1).sqrt() * rr)))


def backward64(s, f, xs, ys, off):
    """Gradients of sum(n dn) + sum(r dr), by autograd through the forward in 64 bits."""
    v = {k: s[k].double().requires_grad_() for k in ("x", "y", "post", "pre")}
    if s["gate"] is not None:
        v["g"] = s["gate"].double().requires_grad_()
    gate = None if s["gate"] is None else v["g"][:, None] if s["kind"] == bs.GATE_TOKEN else v["g"]
    r, n = forward64(s, xs, ys, 1e-6, off, v["x"], v["y"], v["post"], v["pre"], gate)[:2]
    ((n * s["dn"].double()).sum() + (r * s["dr"].double()).sum()).backward()
    return {k: t.grad for k, t in v.items()}


@pytest.mark.parametrize("rows,cols", SHAPES + [(1100, 96), (2300, 40), (700, 7168)])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_gradient(rows, cols, gate):
    """fp32 stream: the saved r is exact, so the gradient is that of the forward by autograd."""
    s = case(rows, cols, torch.float32, gate, 3)
    xs, ys, off = 1.25, 0.5, 1.0
    f = bs.residual_norm(s["x"], s["y"], s["post"], s["pre"], s["gate"], s["kind"], x_scale=xs, y_scale=ys,
                         weight_offset=off)
    got = bs.residual_norm_grad(s["dn"], s["dr"], f["r"], f["rstd_r"], s["pre"], s["y"], f["rstd_y"], s["post"],
                                s["gate"], s["kind"], x_scale=xs, y_scale=ys, weight_offset=off)
    ref = backward64(s, f, xs, ys, off)
    # sizes of the terms of each gradient
    rr, ry = f["rstd_r"].double()[:, None], f["rstd_y"].double()[:, None]
    rh, yh = (f["r"].double() * rr).abs(), (s["y"].double() * ry).abs()
    wp, wq = (s["post"].double() + off).abs(), (s["pre"].double() + off).abs()
    g1 = s["dn"].double().abs() * wq
    # r itself (and so rh) is off by half a step of fp32 and a few operations on its terms
    rmag = forward64(s, xs, ys, 1e-6, off)[4] * rr
    d = s["dr"].double().abs() + rr * (g1 + rh * (g1 * rh).mean(1, keepdim=True)
                                      + rmag * (g1 * rh).mean(1, keepdim=True) + rh * (g1 * rmag).mean(1, keepdim=True))
    close(got["dx"], ref["x"], xs * d)
    g = gate64(s).abs()
    dz = ys * d * g
    g2 = dz * wp
    close(got["dy"], ref["y"], ry * (g2 + yh * (g2 * yh).mean(1, keepdim=True)))
    slots = bs.residual_norm_grad_workspace_bytes(rows, cols) // (8 * cols)
    chain = (rows / slots + slots / 16 + 24) * 2.0 ** -24 + 2.0 ** -17
    close(got["dpre_weight"], ref["pre"], (s["dn"].double().abs() * (rh + rmag)).sum(0), chain)
    close(got["dpost_weight"], ref["post"], (dz * yh).sum(0), chain)
    if gate == "channel":
        close(got["dgate"], ref["g"], (ys * d * yh * wp).sum(0), chain)
    elif gate == "token":
        close(got["dgate"], ref["g"], (ys * d * yh * wp).sum(1))


def test_gradient_against_differences():
    """Central differences of the 64-bit forward along random directions: their own error is of the
    third derivative's order, h^2 = 1e-8 of the size of the terms, below the sums' 1e-5."""
    s = case(6, 200, torch.float32, "channel", 5)
    f = bs.residual_norm(s["x"], s["y"], s["post"], s["pre"], s["gate"], s["kind"])
    got = bs.residual_norm_grad(s["dn"], s["dr"], f["r"], f["rstd_r"], s["pre"], s["y"], f["rstd_y"], s["post"],
                                s["gate"], s["kind"])

    def loss(**more):
        r, n = forward64(s, **more)[:2]
        return float((n * s["dn"].double()).sum() + (r * s["dr"].double()).sum())

    g = torch.Generator(device=DEV).manual_seed(1)
    for name, base, grad in (("x", s["x"], got["dx"]), ("y", s["y"], got["dy"]), ("post", s["post"], got["dpost_weight"]),
                             ("pre", s["pre"], got["dpre_weight"]), ("gate", s["gate"], got["dgate"])):
        v = torch.randn(base.shape, generator=g, device=DEV, dtype=torch.float64)
        h = 1e-4
        diff = (loss(**{name: base.double() + h * v}) - loss(**{name: base.double() - h * v})) / (2 * h)
        size = float((grad.double() * v).abs().sum())
        # dy is rounded to bf16: half a step of each term
        tol = (HALF[grad.dtype] + 2.0 ** -15) * size
        assert abs(diff - float((grad.double() * v).sum())) <= tol, name


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
def test_parts_left_out(stream):
    s = case(5, 136, stream, "none", 7)
    # only the norm before a block
    out = bs.residual_norm(s["x"], pre_weight=s["pre"])
    x = s["x"].double()
    rr = (x.square().mean(1) + 1e-6).rsqrt()
    n = x * rr[:, None] * s["pre"].double()
    assert torch.equal(out["r"], s["x"]) and set(out) == {"r", "n", "rstd_r"}
    close(out["n"], n, n.abs())
    # only the residual sum
    out = bs.residual_norm(s["x"], s["y"], y_scale=0.5)
    r = x + 0.5 * s["y"].double()
    assert set(out) == {"r"}
    close(out["r"], r, x.abs() + s["y"].double().abs())
    # its gradient: no norm on either side
    got = bs.residual_norm_grad(None, s["dr"], y=s["y"], y_scale=0.5, x_scale=2.0)
    assert set(got) == {"dx", "dy"}
    close(got["dx"], 2 * s["dr"].double(), s["dr"].double().abs())
    close(got["dy"], 0.5 * s["dr"].double(), s["dr"].double().abs())
    # the norm before a block alone, nothing else arriving at r
    f = bs.residual_norm(s["x"], pre_weight=s["pre"])
    got = bs.residual_norm_grad(s["dn"], None, f["r"], f["rstd_r"], s["pre"])
    g1, rh, rk = s["dn"].double() * s["pre"].double(), x * rr[:, None], rr[:, None]
    ref = rk * (g1 - rh * (g1 * rh).mean(1, keepdim=True))
    close(got["dx"], ref, rk * (g1.abs() + rh.abs() * (g1 * rh).abs().mean(1, keepdim=True)))


def test_accumulate_no_rows_in_place_and_repeat():
    s = case(300, 264, torch.bfloat16, "channel", 9)
    f = bs.residual_norm(s["x"], s["y"], s["post"], s["pre"], s["gate"], s["kind"])
    args = (s["dn"], s["dr"], f["r"], f["rstd_r"], s["pre"], s["y"], f["rstd_y"], s["post"], s["gate"], s["kind"])
    one = bs.residual_norm_grad(*args)
    two = bs.residual_norm_grad(*args)
    for k in one:
        assert torch.equal(one[k], two[k]), k
    sums = {k: torch.randn_like(one[k]) for k in ("dpre_weight", "dpost_weight", "dgate")}
    want = {k: v + one[k] for k, v in sums.items()}
    bs.residual_norm_grad(*args, accumulate=True, **sums)
    for k in sums:
        assert torch.equal(sums[k], want[k]), k
    # in place: dx over dr, dy over dn, r over x
    dn, dr, x = s["dn"].clone(), s["dr"].clone(), s["x"].clone()
    bs.residual_norm_grad(dn, dr, *args[2:], dx=dr, dy=dn)
    assert torch.equal(dr, one["dx"]) and torch.equal(dn, one["dy"])
    bs.residual_norm(x, s["y"], s["post"], s["pre"], s["gate"], s["kind"], r=x)
    assert torch.equal(x, f["r"])
    # no rows: sums of nothing
    e = {k: s[k][:0] for k in ("x", "y", "dn", "dr")}
    f0 = bs.residual_norm(e["x"], e["y"], s["post"], s["pre"], s["gate"], s["kind"])
    assert f0["r"].shape == (0, 264)
    z = bs.residual_norm_grad(e["dn"], e["dr"], f0["r"], f0["rstd_r"], s["pre"], e["y"], f0["rstd_y"], s["post"],
                              s["gate"], s["kind"])
    for k in ("dpre_weight", "dpost_weight", "dgate"):
        assert not z[k].any(), k


def test_extreme_rows():
    """Rows of zeros (only eps keeps the norm finite), of bf16's largest numbers, and rows with inf and
    NaN, which stay in their own rows."""
    s = case(6, 96, torch.float32, "none", 11)
    s["x"][0], s["y"][0] = 0, 0
    s["x"][1] = 1e18
    s["y"][2] = 1e18
    s["x"][3, 5] = float("inf")
    s["y"][4, 7] = float("nan")
    out = bs.residual_norm(s["x"], s["y"], s["post"], s["pre"])
    assert not out["r"][0].any() and not out["n"][0].any()
    assert float(out["rstd_y"][0]) == pytest.approx(1e3, rel=1e-6)
    keep = [0, 1, 2, 5]
    t = {k: (v[keep] if k in ("x", "y") else v) for k, v in s.items()}
    r, n, ry, rr, mag, w = forward64(t)
    close(out["r"][keep], r, mag)
    close(out["n"][keep], n, mag * rr[:, None] * w.abs() + n.abs())
    assert not torch.isfinite(out["n"][3, 5]) and torch.isnan(out["r"][4]).all()


def test_other_stream_and_graph():
    s = case(37, 640, torch.bfloat16, "token", 13)
    args = (s["x"], s["y"], s["post"], s["pre"], s["gate"], s["kind"])
    want = bs.residual_norm(*args)
    grad = (s["dn"], s["dr"], want["r"], want["rstd_r"], s["pre"], s["y"], want["rstd_y"], s["post"], s["gate"],
            s["kind"])
    back = bs.residual_norm_grad(*grad)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = bs.residual_norm(*args)
    side.synchronize()
    for k in want:
        assert torch.equal(got[k], want[k]), k
    out = {k: torch.empty_like(v) for k, v in want.items()}
    gout = {k: torch.empty_like(v) for k, v in back.items()}
    ws = torch.empty(bs.residual_norm_grad_workspace_bytes(37, 640), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bs.residual_norm(*args, **out)
        bs.residual_norm_grad(s["dn"], s["dr"], out["r"], out["rstd_r"], s["pre"], s["y"], out["rstd_y"], s["post"],
                              s["gate"], s["kind"], workspace=ws, **gout)
    for seed in (1, 2, 3):
        new = case(37, 640, torch.bfloat16, "token", 20 + seed)
        for k in ("x", "y", "dn", "dr"):
            s[k].copy_(new[k])
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        want = bs.residual_norm(*args)
        back = bs.residual_norm_grad(s["dn"], s["dr"], want["r"], want["rstd_r"], s["pre"], s["y"], want["rstd_y"],
                                     s["post"], s["gate"], s["kind"])
        for k in out:
            assert torch.equal(out[k], want[k]), k
        for k in gout:
            assert torch.equal(gout[k], back[k]), k
