"""layernorm and layernorm_bwd, and the norms' 8-bit outputs with block scales, on the GPU against plain 64-bit
forms."""
import pytest
import torch

import dense_gemm_matrix_amd as dg
from tests.feedforward_ref import H, blocks, layer64, layer_grad64, rounded, spread
from tests.linear_ref import F8, U, gap_kept, padded, sentinel, within
from tests.test_gpu_norm import DTS, SIZES, norm64, rows, rstd_err

pytestmark = pytest.mark.gpu

EPS = 1e-5
WIDTHS = [(256, 2050), (257, 2050), (257, 4100), (256, 8190), (257, 8190)]  # either side of one row per CU


def vector(n, seed, base=0.0):
    return rows(1, n, torch.float32, seed)[0] + base


def nans(*shape):
    return torch.full(shape, float("nan"), device="cuda")


@pytest.mark.parametrize("dt", DTS, ids=str)
@pytest.mark.parametrize("size", SIZES + WIDTHS + [(2, 20000), (2, 32768)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("res, bias, shift", [(False, True, 0.0), (True, False, 0.0), (True, True, 50.0)])
def test_forward(dt, size, res, bias, shift):
    M, N = size
    X, R = (rows(M, N, torch.float32, 1) + shift).to(dt), rows(M, N, dt, 2) if res else None
    w, b = vector(N, 3, 1.0), vector(N, 4) if bias else None
    Y, S, m, r = sentinel(M, N, dt), sentinel(M, N, dt, 2), nans(M), nans(M)
    dg.layernorm(padded(X, dt, 1), w.cuda(), None if b is None else b.cuda(), Y,
                 residual=None if R is None else padded(R, dt, 2), total=S, mean=m, rstd=r, eps=EPS)
    torch.cuda.synchronize()
    (s, es), (mean, em), (rstd, er), (y, ey) = layer64(X, R, w, b, EPS)
    within(S, s, rounded(es, s, dt))
    within(m, mean, em)
    within(r, rstd, er)
    within(Y, y, rounded(ey, y, dt))
    assert gap_kept(Y) and gap_kept(S)


@pytest.mark.parametrize("dt", DTS, ids=str)
@pytest.mark.parametrize("size", SIZES + WIDTHS + [(2, 32768)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("kind", ["row", "block", "block rows apart", "rms block"])
def test_forward_f8(dt, size, kind):
    M, N = size
    X, R = rows(M, N, dt, 5), rows(M, N, dt, 6)
    w, b = vector(N, 7, 1.0), vector(N, 8)
    Y, S = sentinel(M, N, F8), sentinel(M, N, dt)
    if kind == "row":
        sc = nans(M)
    elif kind == "block rows apart":  # a row's scales next to each other, rows padded
        sc = nans(M, blocks(N) + 3)[:, :blocks(N)]
    else:
        sc = nans(blocks(N), M).t()
    if kind == "rms block":
        dg.rmsnorm(padded(X, dt), w.cuda(), Y, residual=padded(R, dt), total=S, scale=sc, eps=EPS)
        y = norm64(X, R, w, EPS)[2]
        ey = (rstd_err(N) + 6 * H) * y.abs()
    else:
        dg.layernorm(padded(X, dt), w.cuda(), b.cuda(), Y, residual=padded(R, dt), total=S, scale=sc, eps=EPS)
        y, ey = layer64(X, R, w, b, EPS)[3]
    torch.cuda.synchronize()
    if kind == "row":
        want, err = y.abs().amax(1, keepdim=True) / 448, ey.amax(1, keepdim=True) / 448
        each = lambda t: t.reshape(M, 1).double().expand(M, N)  # noqa: E731
        got = sc.cpu()[:, None]
    else:
        part = torch.zeros(M, blocks(N) * 128, dtype=torch.float64)
        part[:, :N] = y.abs()
        pe = torch.zeros_like(part)
        pe[:, :N] = ey
        want, err = part.view(M, -1, 128).amax(2) / 448, pe.view(M, -1, 128).amax(2) / 448
        each = lambda t: spread(t, 1, M, N)  # noqa: E731
        got = sc.cpu()
    within(got, want.clamp_min(2.0 ** -100), err + 2 * H * want + 2.0 ** -120)
    # A code stands for a value within half a step of e4m3 (2^-4 relative, 2^-10 scales) of y's fp32 value.
    v = Y.cpu().double() * each(got)
    within(v, y, ey + (2.0 ** -4 + 4 * H) * (y.abs() + ey) + 2.0 ** -10 * each(got) * (1 + 4 * H))
    assert gap_kept(Y)
    # The largest magnitude of a block that has one takes the largest code (two of e4m3's half steps of fp32 are far less).
    if kind == "block":
        codes = torch.zeros(M, blocks(N) * 128)
        codes[:, :N] = Y.cpu().float().abs()
        assert (codes.view(M, -1, 128).amax(2) == 448).all()


def test_rows_in_place():
    M, N = 37, 1000
    X, R = rows(M, N, torch.bfloat16, 1), rows(M, N, torch.bfloat16, 2)
    w, b = vector(N, 3, 1.0).cuda(), vector(N, 4).cuda()
    want = dg.layer_norm(padded(X, X.dtype), w, b, residual=padded(R, R.dtype), keep=True)
    x, r = padded(X, X.dtype), padded(R, R.dtype)
    dg.layernorm(x, w, b, x, residual=r, total=r, eps=EPS)
    torch.cuda.synchronize()
    assert torch.equal(x, want["Y"]) and torch.equal(r, want["total"])


def test_nonfinite_rows_keep_to_themselves():
    """A row with an infinity or a NaN gives NaN (its scales too), its neighbours what they give without it."""
    M, N = 9, 700
    X = rows(M, N, torch.float32, 5)
    w, b = vector(N, 3, 1.0).cuda(), vector(N, 4).cuda()
    ref, ref8 = dg.layer_norm(X.cuda(), w, b), dg.layer_norm(X.cuda(), w, b, f8="block")
    for bad in (float("inf"), float("-inf"), float("nan")):
        Z = X.clone()
        Z[4, 300] = bad
        y, y8 = dg.layer_norm(Z.cuda(), w, b, keep=True), dg.layer_norm(Z.cuda(), w, b, f8="block")
        keep = torch.arange(M) != 4
        assert torch.equal(y["Y"][keep], ref["Y"][keep]) and torch.equal(y8["scale"][keep], ref8["scale"][keep])
        assert torch.equal(y8["Y"][keep].float(), ref8["Y"][keep].float())
        assert y["Y"][4].isnan().all() and y["rstd"][4].isnan() and y8["scale"][4].isnan().all()


def test_constant_rows():
    """A row without variance: y is the bias, its 8-bit scales the bias' own, rstd eps^-1/2."""
    X = torch.full((5, 260), 3.0).cuda()
    b = vector(260, 4)
    out = dg.layer_norm(X, vector(260, 3).cuda(), b.cuda(), keep=True, eps=1e-4)
    assert torch.equal(out["Y"].cpu(), b.expand(5, 260))
    within(out["rstd"], torch.full((5,), 100.0, dtype=torch.float64), torch.full((5,), 100 * 8 * H, dtype=torch.float64))
    zero = dg.layer_norm(X, vector(260, 3).cuda(), f8="block")
    assert (zero["Y"].float() == 0).all() and (zero["scale"] == 2.0 ** -100).all()


BWD_SIZES = [s for s in SIZES] + [(700, 64), (300, 257), (515, 1030), (600, 2048), (1100, 96), (270, 4100)]


@pytest.mark.parametrize("dt", DTS, ids=str)
@pytest.mark.parametrize("size", BWD_SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("res", [False, True])
def test_backward(dt, size, res):
    M, N = size
    dY, S = rows(M, N, dt, 1), (rows(M, N, torch.float32, 2) + 3.0).to(dt)
    dS = rows(M, N, dt, 3) if res else None
    w = vector(N, 4, 1.0)
    mean = S.float().mean(1)
    rstd = (S.float().var(1, unbiased=False) + EPS).rsqrt()
    dX, dw, db = sentinel(M, N, dt, 2), nans(N), nans(N)
    ws = torch.empty(dg.layernorm_bwd_workspace(M, N), dtype=torch.uint8, device="cuda")
    dg.layernorm_bwd(padded(dY, dt, 1), padded(S, dt), w.cuda(), mean.cuda(), rstd.cuda(), dX,
                     dtotal=None if dS is None else padded(dS, dt, 3), dweight=dw, dbias=db, workspace=ws)
    torch.cuda.synchronize()
    (dx, ex), (w64, ew), (b64, eb) = layer_grad64(dY, S, w, mean, rstd, dS)
    within(dX, dx, rounded(ex, dx, dt))
    within(dw, w64, ew + 1e-30)
    within(db, b64, eb + 1e-30)
    assert gap_kept(dX)


def test_backward_is_the_gradient():
    """Against differences of the forward definition in 64 bits."""
    M, N, h = 3, 40, 1e-6
    X, dY = rows(M, N, torch.float32, 1).double(), rows(M, N, torch.float32, 2).double()
    w, b = vector(N, 3, 1.0).double(), vector(N, 4).double()

    def loss(x, w_, b_):
        d = x - x.mean(1, keepdim=True)
        return (dY * (d * (d.square().mean(1, keepdim=True) + EPS).rsqrt() * w_ + b_)).sum()

    out = dg.layer_norm(X.float().cuda(), w.float().cuda(), b.float().cuda(), keep=True, eps=EPS)
    dx, dw, db = dg.layer_norm_backward(dY.float().cuda(), X.float().cuda(), w.float().cuda(), out["mean"], out["rstd"])
    x0, w0 = X.float().double(), w.float().double()
    for i, j in [(0, 0), (1, 17), (2, 39)]:
        e = torch.zeros_like(x0)
        e[i, j] = h
        num = (loss(x0 + e, w0, b) - loss(x0 - e, w0, b)) / (2 * h)
        assert abs(float(num) - float(dx[i, j])) < 1e-5  # fp32's 40-term sums, and h^2
        f = torch.zeros_like(w0)
        f[j] = h
        assert abs(float((loss(x0, w0 + f, b) - loss(x0, w0 - f, b)) / (2 * h)) - float(dw[j])) < 1e-5
        assert abs(float((loss(x0, w0, b + f) - loss(x0, w0, b - f)) / (2 * h)) - float(db[j])) < 1e-5


def test_backward_parts_and_in_place():
    """Each gradient asked for alone, dX over dY and over dtotal: the same bits."""
    M, N = 300, 520
    dt = torch.bfloat16
    dY, S, dS = rows(M, N, dt, 1).cuda(), rows(M, N, dt, 2).cuda(), rows(M, N, dt, 3).cuda()
    w = vector(N, 4, 1.0).cuda()
    mean, rstd = S.float().mean(1), (S.float().var(1, unbiased=False) + EPS).rsqrt()
    ws = torch.empty(dg.layernorm_bwd_workspace(M, N), dtype=torch.uint8, device="cuda")
    dX, dw, db = torch.empty_like(dY), nans(N), nans(N)
    dg.layernorm_bwd(dY, S, w, mean, rstd, dX, dtotal=dS, dweight=dw, dbias=db, workspace=ws)
    for kw in (dict(), dict(dweight=nans(N)), dict(dbias=nans(N))):
        x = torch.empty_like(dY)
        dg.layernorm_bwd(dY, S, w, mean, rstd, x, dtotal=dS, workspace=ws if kw else None, **kw)
        assert torch.equal(x, dX)
        for k, v in kw.items():
            assert torch.equal(v, dw if k == "dweight" else db)
    for over in ("dY", "dS"):
        y, s = dY.clone(), dS.clone()
        dg.layernorm_bwd(y, S, w, mean, rstd, y if over == "dY" else s, dtotal=s)
        assert torch.equal(y if over == "dY" else s, dX)


def test_empty():
    w = torch.ones(8, device="cuda")
    e = torch.empty(0, 8, device="cuda")
    out = dg.layer_norm(e, w, w, f8="block")
    assert out["Y"].shape == (0, 8) and out["scale"].shape == (0, 1)
    dx, dw, db = dg.layer_norm_backward(e, e, w, torch.empty(0, device="cuda"), torch.empty(0, device="cuda"))
    assert dx.shape == (0, 8) and (dw == 0).all() and (db == 0).all()


def test_refusals():
    X, w = torch.zeros(4, 8, device="cuda"), torch.ones(8, device="cuda")
    Y8 = torch.empty(4, 16, dtype=F8, device="cuda")[:, :8]
    v4 = torch.ones(4, device="cuda")
    for args, kw in [((X, w, None, Y8), {}), ((X, w, None, X), dict(scale=v4)),
                     ((X, w, w[:4], torch.empty_like(X)), {}), ((X, None, None, X), {}),
                     ((X, w, None, Y8), dict(scale=torch.ones(4, 2, device="cuda"))),
                     ((X, w, None, Y8), dict(scale=torch.ones(3, 1, device="cuda"))),
                     ((X, w, None, X), dict(mean=w)), ((X.cpu(), w, None, X), {})]:
        with pytest.raises((ValueError, TypeError)):
            dg.layernorm(*args, **kw)
    with pytest.raises(dg.DgemmError):
        dg.layernorm(X, w, None, X, eps=-1.0)
    with pytest.raises(dg.DgemmError):  # scales on top of each other
        dg.layernorm(torch.zeros(4, 256, device="cuda"), torch.ones(256, device="cuda"), None,
                     torch.empty(4, 256, dtype=F8, device="cuda"), scale=v4[:1].expand(4, 2))
    with pytest.raises(dg.DgemmError):
        dg.layernorm_bwd(X, X, w, v4, v4, torch.empty_like(X), dweight=torch.empty_like(w))  # no workspace
    with pytest.raises(ValueError):
        dg.rmsnorm(torch.zeros(4, 256, device="cuda"), torch.ones(256, device="cuda"),
                   torch.empty(4, 256, dtype=F8, device="cuda"), scale=torch.ones(4, 2, device="cuda"))


def test_captured_and_on_another_stream():
    M, N = 200, 1500
    dt = torch.float16
    x, r = rows(M, N, dt, 1).cuda(), rows(M, N, dt, 2).cuda()
    x, r = padded(x.cpu(), dt), padded(r.cpu(), dt)
    w, b = vector(N, 3, 1.0).cuda(), vector(N, 4).cuda()
    side = torch.cuda.Stream()

    def step(stream=None):
        o = dg.layer_norm(x, w, b, residual=r, keep=True, stream=stream)
        q = dg.layer_norm(x, w, b, residual=r, f8="block", stream=stream)
        g = dg.layer_norm_backward(o["Y"], o["total"], w, o["mean"], o["rstd"], dtotal=r, stream=stream)
        return [o["Y"], o["total"], o["mean"], o["rstd"], q["Y"].view(torch.uint8), q["scale"], *g]

    want = [t.clone() for t in step()]
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        x.copy_(rows(M, N, dt, 20 + i))
        want = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(out, want)), i
