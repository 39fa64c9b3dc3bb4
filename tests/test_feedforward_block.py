"""A feed-forward block as a program runs it, forward and backward: layer norm with the residual, gated projection,
projection back and residual; the operators hand each other their results.  Against the same formulas in 64 bits
throughout: every stage's error bound is carried through the stages behind it."""
import pytest
import torch

import dense_gemm_matrix_amd as dg
from tests.feedforward_ref import H, block_bound, block_product64, layer64, quant_block64, rounded
from tests.linear_ref import F8, SLOPE, act64, act_grad64, out_bound, padded, sum_bound, within

gpu = pytest.mark.gpu

CURVE = 1.2    # above the largest |act''|: GELU's 0.8, SiLU's 0.5
SECOND = 1.05  # products of two of the errors below, all far under 1 / 20 of what they multiply
EPS = 1e-5


def block_inputs(M, D, F, dt, seed):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s, by=1.0: (torch.randn(*s, generator=g) * by).to(dt)  # noqa: E731
    t = dict(x=rnd(M, D), r=rnd(M, D), Bg=rnd(D, F, by=D ** -0.5), Bu=rnd(D, F, by=D ** -0.5),
             Bd=rnd(F, D, by=F ** -0.5), dO=rnd(M, D))
    v = dict(w=torch.rand(D, generator=g) + 0.5, b=torch.randn(D, generator=g), bg=torch.randn(F, generator=g),
             bu=torch.randn(F, generator=g))
    return t, v


def block(t, v, act):
    """Forward and backward with the public entry points."""
    n = dg.layer_norm(t["x"], v["w"], v["b"], residual=t["r"], keep=True, eps=EPS)
    c, G, U = dg.linear_gated(n["Y"], t["Bg"], t["Bu"], bias_g=v["bg"], bias_u=v["bu"], act=act, keep_preact=True)
    o = dg.linear(c, t["Bd"], residual=n["total"])
    dc, dBd, _ = dg.linear_backward(c, t["Bd"], t["dO"])
    dy, dBg, dBu, dbg, dbu = dg.linear_gated_backward(n["Y"], t["Bg"], t["Bu"], dc, G, U, act=act, bias=True)
    dx, dw, db = dg.layer_norm_backward(dy, n["total"], v["w"], n["mean"], n["rstd"], dtotal=t["dO"])
    return dict(o=o, dBd=dBd, dBg=dBg, dBu=dBu, dbg=dbg, dbu=dbu, dx=dx, dw=dw, db=db)


def block64(t, v, act, dt):
    """name -> (value, bound)."""
    d = {k: x.double() for k, x in {**t, **v}.items()}
    M, D = d["x"].shape
    F = d["Bg"].shape[1]
    f32 = torch.float32
    (s, es), (mean, em), (rstd, er), (y, ey) = layer64(t["x"], t["r"], v["w"], v["b"], EPS)
    # the operators hand on roundings to the matrices' type; the statistics are of the fp32 sums
    es_st, ey = rounded(es, s, dt), rounded(ey, y, dt)
    z = {}
    for k, B, b in (("g", "Bg", "bg"), ("u", "Bu", "bu")):
        p, S = y @ d[B] + d[b], (y.abs() + ey) @ d[B].abs() + d[b].abs()
        z[k] = (p, ey @ d[B].abs() + sum_bound(D, S))
    (g, eg), (u, eu) = z["g"], z["u"]
    a, ea = act64(g, act), SLOPE * eg + 32 * H * g.abs()
    c = a * u
    ec = rounded(SECOND * (u.abs() * ea + a.abs() * eu) + 2 * H * c.abs(), c, dt)
    eg, eu = rounded(eg, g, dt), rounded(eu, u, dt)  # as they are kept for the backward pass
    o = c @ d["Bd"] + s
    eo = ec @ d["Bd"].abs() + sum_bound(F, (c.abs() + ec) @ d["Bd"].abs()) + es_st + H * o.abs()
    out = {"o": (o, rounded(eo, o, dt))}
    dO = d["dO"]
    dc, edc = dO @ d["Bd"].t(), sum_bound(D, dO.abs() @ d["Bd"].abs().t())
    edc = rounded(edc, dc, dt)
    out["dBd"] = (c.t() @ dO, ec.t() @ dO.abs() + sum_bound(M, (c.abs() + ec).t() @ dO.abs()))
    sl = act_grad64(g, act)
    zg, zu = dc * u * sl, dc * a
    ezg = SECOND * (edc * (u * sl).abs() + dc.abs() * eu * sl.abs() + (dc * u).abs() * (CURVE * eg + 32 * SLOPE * H))
    ezu = SECOND * (edc * a.abs() + dc.abs() * (SLOPE * eg + 32 * H * g.abs()))
    ezg, ezu = ezg + 3 * H * zg.abs(), ezu + 3 * H * zu.abs()
    for k, x, e in (("dbg", zg, ezg), ("dbu", zu, ezu)):
        out[k] = (x.sum(0), e.sum(0) + (M + 2) * H * (x.abs() + e).sum(0))
    ezg, ezu = rounded(ezg, zg, dt), rounded(ezu, zu, dt)
    for k, x, e in (("dBg", zg, ezg), ("dBu", zu, ezu)):
        ab = SECOND * (ey.t() @ x.abs() + y.abs().t() @ e)
        out[k] = (y.t() @ x, ab + sum_bound(M, (y.abs() + ey).t() @ (x.abs() + e)))
    dy = zg @ d["Bg"].t() + zu @ d["Bu"].t()
    edy = ezg @ d["Bg"].abs().t() + ezu @ d["Bu"].abs().t()
    edy = edy + sum_bound(2 * F, (zg.abs() + ezg) @ d["Bg"].abs().t() + (zu.abs() + ezu) @ d["Bu"].abs().t())
    edy = rounded(edy, dy, dt)
    r, er, mean, em = rstd[:, None], er[:, None], mean[:, None], em[:, None]
    xh, gy = (s - mean) * r, dy * d["w"]
    exh = SECOND * ((es_st + em) * r + xh.abs() * er / r)
    egy = edy * d["w"].abs()
    mg, mgx = gy.mean(1, keepdim=True), (gy * xh).mean(1, keepdim=True)
    inner = gy - mg - xh * mgx
    mean1 = lambda x: x.mean(1, keepdim=True)  # noqa: E731
    emgx = mean1(egy * xh.abs() + gy.abs() * exh)
    e = r * SECOND * (egy + mean1(egy) + xh.abs() * emgx + exh * mgx.abs()) + er * inner.abs()
    e = e + r * ((D + 4) * H * mean1(gy.abs()) + xh.abs() * (D + 8) * H * mean1((gy * xh).abs())
                 + 6 * H * (gy.abs() + mg.abs() + (xh * mgx).abs()))
    dx = r * inner + dO
    out["dx"] = (dx, SECOND * e + 3 * H * (dx.abs() + dO.abs()))
    t1 = (dy * xh).abs() + edy * xh.abs() + dy.abs() * exh
    out["dw"] = ((dy * xh).sum(0), SECOND * (edy * xh.abs() + dy.abs() * exh).sum(0) + (M + 5) * H * t1.sum(0))
    out["db"] = (dy.sum(0), edy.sum(0) + (M + 2) * H * (dy.abs() + edy).sum(0))
    return {k: (x, b if k in ("o", "dbg", "dbu", "dw", "db") else rounded(b, x, dt) if dt != f32 else b + H * x.abs())
            for k, (x, b) in out.items()}


def test_bounds_see_a_mistake():
    """With another activation, without the residual's way or with the gates exchanged, every result that depends on
    it is out of its bound."""
    t, v = block_inputs(100, 264, 520, torch.float32, seed=3)
    want = block64(t, v, "silu", torch.float32)

    def seen(other):
        return {k for k, (x, b) in want.items() if ((other[k][0] - x).abs() > b).any()}

    assert seen(want) == set()
    assert seen(block64(t, v, "gelu", torch.float32)) == set(want)
    assert seen(block64({**t, "r": torch.zeros_like(t["r"])}, v, "silu", torch.float32)) == set(want)
    assert seen(block64({**t, "Bg": t["Bu"], "Bu": t["Bg"]}, v, "silu", torch.float32)) == set(want)


@gpu
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("shape", [(1, 200, 264), (13, 72, 136), (100, 264, 520), (400, 520, 136)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_block_forward_and_backward(dt, shape, act):
    t, v = block_inputs(*shape, dt, seed=shape[0])
    got = block({k: padded(x, dt) for k, x in t.items()}, {k: x.cuda() for k, x in v.items()}, act)
    want = block64(t, v, act, dt)
    for k, (x, b) in want.items():
        try:
            within(got[k], x, b)
        except AssertionError as e:
            raise AssertionError(f"{k}: {e}")


@gpu
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=str)
def test_block_captured_and_on_a_stream(dt):
    """The whole of it on a side stream and as a replayed graph: the bits of the plain run, for new inputs each time."""
    M, D, F = 150, 264, 520
    t, v = block_inputs(M, D, F, dt, seed=1)
    t, v = {k: padded(x, dt) for k, x in t.items()}, {k: x.cuda() for k, x in v.items()}
    want = {k: x.clone() for k, x in block(t, v, "silu").items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = block(t, v, "silu")
    side.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(t, v, "silu")
    for i in range(4):
        new, nv = block_inputs(M, D, F, dt, seed=10 + i)
        for k, x in new.items():
            t[k].copy_(x)
        for k, x in nv.items():
            v[k].copy_(x)
        want = {k: x.clone() for k, x in block(t, v, "silu").items()}
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], want[k]) for k in want), i


@gpu
@pytest.mark.parametrize("M", [1, 30, 300])
@pytest.mark.parametrize("norm", ["layer", "rms"])
def test_norm_to_8_bit_projection(M, norm):
    """A norm that writes 8 bits with a scale per row and 128 columns, and the projection that reads them."""
    D, N = 520, 264
    g = torch.Generator().manual_seed(M)
    x, r = (torch.randn(M, D, generator=g).bfloat16() for _ in range(2))
    w, b = torch.rand(D, generator=g) + 0.5, torch.randn(D, generator=g)
    W = (torch.randn(D, N, generator=g) / D ** 0.5).bfloat16()
    xd, rd = padded(x, x.dtype), padded(r, r.dtype)
    if norm == "layer":
        n = dg.layer_norm(xd, w.cuda(), b.cuda(), residual=rd, f8="block")
        y, ey = layer64(x, r, w, b, EPS)[3]
    else:
        n = dg.rms_norm(xd, w.cuda(), residual=rd, f8="block", eps=1e-6)
        s = x.double() + r.double()
        rr = (s.square().mean(1, keepdim=True) + 1e-6).rsqrt()
        y = s * rr * w.double()
        ey = (D + 8) * H * y.abs()
    wq, ws = dg.quantize_f8_block(padded(W, W.dtype), rows=128, transpose=True)
    q, sc = quant_block64(W.t(), 128)
    assert torch.equal(wq.cpu().double(), q) and torch.equal(ws.cpu(), sc)
    o = dg.matmul_f8_block(n["Y"], wq, n["scale"], ws, bias=None, residual=None)
    Z, S, drop = block_product64(n["Y"].cpu(), wq.cpu(), n["scale"].cpu(), ws.cpu(), 128)
    within(o, Z, out_bound(Z, Z, block_bound(D, S) + drop, None, torch.bfloat16, "none"))
    # what the codes stand for is the norm's result within half a step of e4m3: 2^-4 of a value, or of the block's
    # smallest normal code, and the scale's rounding
    code = n["Y"].cpu().double() * n["scale"].cpu().double().repeat_interleave(128, 1)[:, :D]
    sc = n["scale"].cpu().double().repeat_interleave(128, 1)[:, :D]
    within(code, y, 1.01 * ey + (2.0 ** -4 + 4 * H) * (y.abs() + ey) + 2.0 ** -10 * sc * 1.01)
