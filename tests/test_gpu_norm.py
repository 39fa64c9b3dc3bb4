"""rmsnorm, rmsnorm_bwd and quant_f8 on the GPU against plain 64-bit forms."""
import pytest
import torch

import dense_gemm_matrix_amd as dg
from tests.linear_ref import F8, TINY, U, gap_kept, padded, quant64, sentinel, within

pytestmark = pytest.mark.gpu

DTS = [torch.float32, torch.bfloat16, torch.float16]
EPS = 1e-5
# every variant of threads per row and columns per lane, odd sizes among them
SIZES = [(1, 1), (3, 7), (37, 64), (70, 128), (1, 130), (19, 250), (5, 512), (9, 513), (2, 1024), (4, 1030), (3, 2048), (6, 3001), (2, 4096), (3, 8190),
         (2, 9001), (2, 16384)]


def rows(M, N, dt, seed, scale=1.0):
    return (torch.randn(M, N, generator=torch.Generator().manual_seed(seed)) * scale).to(dt)


def norm64(X, R, w, eps=EPS):
    s = X.double() if R is None else X.double() + R.double()
    rstd = (s.square().mean(1) + eps).rsqrt()
    return s, rstd, s * rstd[:, None] * w.double()


def rstd_err(N):
    """Relative error of the fp32 rstd: half of the sum of squares' (N half steps,
    and two for the residual's addition that each square doubles), the mean's and
    eps' two roundings halved, and rsqrt's 2 ulps."""
    return ((N + 4) / 2 + 1 + 4) * 2.0 ** -24


@pytest.mark.parametrize("dt", DTS, ids=str)
@pytest.mark.parametrize("size", SIZES + [(2, 20000), (2, 32768)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("res", [False, True])
def test_forward(dt, size, res):
    M, N = size
    X, R = rows(M, N, dt, 1), rows(M, N, dt, 2) if res else None
    w = rows(1, N, torch.float32, 3)[0] + 1.0
    Y, S, r = sentinel(M, N, dt), sentinel(M, N, dt, 2), torch.full((M,), float("nan"), device="cuda")
    dg.rmsnorm(padded(X, dt, 1), w.cuda(), Y, residual=None if R is None else padded(R, dt, 2), total=S, rstd=r,
               eps=EPS)
    torch.cuda.synchronize()
    s, rstd, y = norm64(X, R, w)
    e = rstd_err(N)
    within(S, s, 2.0 ** -24 * s.abs() + U[dt] * s.abs() * (1 + 2.0 ** -24) + TINY[dt])
    within(r, rstd, e * rstd)
    b = (e + 4 * 2.0 ** -24) * y.abs()
    within(Y, y, b + U[dt] * (y.abs() + b) + TINY[dt])
    assert gap_kept(Y) and gap_kept(S)


@pytest.mark.parametrize("dt", DTS, ids=str)
@pytest.mark.parametrize("size", SIZES + [(2, 32768)], ids=lambda s: "x".join(map(str, s)))
def test_forward_f8(dt, size):
    M, N = size
    X, R = rows(M, N, dt, 4), rows(M, N, dt, 5)
    w = rows(1, N, torch.float32, 6)[0] + 1.0
    Y, S, sc = sentinel(M, N, F8), sentinel(M, N, dt), torch.full((M,), float("nan"), device="cuda")
    dg.rmsnorm(padded(X, dt), w.cuda(), Y, residual=padded(R, dt), total=S, scale=sc, eps=EPS)
    torch.cuda.synchronize()
    _, _, y = norm64(X, R, w)
    e = rstd_err(N) + 6 * 2.0 ** -24
    scale = (y.abs().amax(1) / 448).clamp_min(2.0 ** -100)
    within(sc, scale, 2 * e * scale)
    # the value a code stands for is off by half a step of e4m3, 2^-4 relative or
    # 2^-10 scales absolute, and by what the fp32 value and scale are off
    v = Y.cpu().double() * sc.cpu().double()[:, None]
    within(v, y, (2.0 ** -4 + 4 * e) * y.abs() + 2.0 ** -10 * (1 + 4 * e) * scale[:, None])
    assert gap_kept(Y)


@pytest.mark.parametrize("dt", DTS, ids=str)
@pytest.mark.parametrize("size", SIZES + [(2, 32768), (70, 130)], ids=lambda s: "x".join(map(str, s)))
def test_quantizer_is_exact(dt, size):
    """Rows and columns: the scale is the fp32 quotient, the codes the nearest
    values of the exact quotients by it."""
    M, N = size
    X = rows(M, N, dt, 7, 3.0)
    X[0] = 0
    for tr in (False, True):
        Xr = X.t() if tr else X
        Q, sc = sentinel(*Xr.shape, F8), torch.full((Xr.shape[0],), float("nan"), device="cuda")
        if tr and N > 10000:
            continue
        dg.quant_f8(padded(X, dt, 1), Q, sc, transpose=tr)
        torch.cuda.synchronize()
        scale = (Xr.float().abs().amax(1) / torch.tensor(448.0)).clamp_min(2.0 ** -100)
        assert torch.equal(sc.cpu(), scale)
        q = (Xr.float() / scale[:, None]).clamp(-448, 448)
        assert torch.equal(Q.cpu().float(), q.to(F8).float())
        assert gap_kept(Q)


def test_quantizer_ties_and_small_rows():
    """Values halfway between codes go to the even one; rows of tiny values, of
    zeros and of one column have a finite scale."""
    codes = torch.arange(0x7f, dtype=torch.uint8).view(F8).float()
    mid = (codes[1:] + codes[:-1]) / 2
    x = torch.cat([mid, -mid, torch.tensor([448.0])])[None]
    Q, sc = dg.quantize_f8(padded(x, torch.float32))
    assert float(sc) == 1.0 and torch.equal(Q.cpu().float(), x.to(F8).float())
    for v in (0.0, 1e-38, -1e-45, 2.0 ** -100 * 448, 3e38):
        Q, sc = dg.quantize_f8(padded(torch.full((1, 5), v), torch.float32))
        assert torch.isfinite(sc).all() and torch.isfinite(Q.float()).all()
        back = Q.float() * sc[:, None]
        assert float((back - v).abs().max()) <= 2.0 ** -4 * abs(v) + 2.0 ** -110


def test_nonfinite_rows_have_no_scale():
    for bad in (float("inf"), float("-inf"), float("nan")):
        x = rows(6, 70, torch.float32, 8)
        x[2, 69] = bad
        Q, sc = dg.quantize_f8(padded(x, torch.float32))
        assert torch.isnan(sc[2]) and torch.isfinite(sc[[0, 1, 3, 4, 5]]).all()
        Q, sc = dg.quantize_f8(padded(x, torch.float32), transpose=True)
        assert torch.isnan(sc[69]) and torch.isfinite(sc[:69]).all()
        got = dg.rms_norm(padded(x, torch.float32), torch.ones(70, device="cuda"), f8=True)
        assert torch.isnan(got["scale"][2]) and torch.isfinite(got["scale"][[0, 1, 3, 4, 5]]).all()


def test_rows_of_zeros_and_in_place():
    """A row of zeros: rstd = eps^-1/2 and outputs 0.  S and Y may be the inputs."""
    X, R = rows(5, 1030, torch.bfloat16, 9), rows(5, 1030, torch.bfloat16, 10)
    X[3] = 0
    R[3] = 0
    w = torch.rand(1030).cuda() + 0.5
    want = dg.rms_norm(padded(X, torch.bfloat16), w, residual=padded(R, torch.bfloat16), keep=True)
    assert bool((want["Y"][3] == 0).all()) and abs(float(want["rstd"][3]) - 1e3) <= 1e-3
    Xd, Rd = padded(X, torch.bfloat16), padded(R, torch.bfloat16)
    dg.rmsnorm(Xd, w, Xd, residual=Rd, total=Rd)
    assert torch.equal(Xd, want["Y"]) and torch.equal(Rd, want["total"])


def bwd64(dY, S, w, rstd, dS):
    dY, S, w, r = dY.double(), S.double(), w.double(), rstd.double()[:, None]
    h, g = S * r, dY * w
    mean = (g * h).mean(1, keepdim=True)
    dX = r * (g - h * mean)
    return (dX if dS is None else dX + dS.double()), (dY * h).sum(0), h, g, mean


@pytest.mark.parametrize("dt", DTS, ids=str)
@pytest.mark.parametrize("size", SIZES + [(600, 40), (1100, 1040), (530, 4096)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("res", [False, True])
def test_backward(dt, size, res):
    M, N = size
    dY, S = rows(M, N, dt, 11), rows(M, N, dt, 12)
    dS = rows(M, N, dt, 13) if res else None
    w = rows(1, N, torch.float32, 14)[0] + 1.0
    rstd = (S.double().square().mean(1) + EPS).rsqrt().float()
    dX, dw = sentinel(M, N, dt), torch.full((N,), float("nan"), device="cuda")
    ws = torch.full((dg.rmsnorm_bwd_workspace(M, N),), 0x7f, dtype=torch.uint8, device="cuda")
    dg.rmsnorm_bwd(padded(dY, dt, 1), padded(S, dt), w.cuda(), rstd.cuda(), dX,
                   dtotal=None if dS is None else padded(dS, dt, 2), dweight=dw, workspace=ws)
    torch.cuda.synchronize()
    ref, dw64, h, g, mean = bwd64(dY, S, w, rstd, dS)
    r = rstd.double()[:, None]
    # the mean's sum: N half steps of absolute products and three per product
    em = (N + 4) * 2.0 ** -24 * (g * h).abs().mean(1, keepdim=True)
    b = r * (4 * 2.0 ** -24 * (g.abs() + (h * mean).abs()) + h.abs() * em) + 2 * 2.0 ** -24 * ref.abs()
    within(dX, ref, b + U[dt] * (ref.abs() + b) + TINY[dt])
    within(dw, dw64, (M + 4) * 2.0 ** -24 * (dY.double() * h).abs().sum(0) + 2.0 ** -149)
    assert gap_kept(dX)


def test_backward_against_differences():
    """The gradient of sum(v o Y) + sum(u o S) by central differences in 64 bits,
    along random directions; the kernel's fp32 error is within 1e-5 of the sum of
    absolute terms (rows of 40)."""
    M, N = 6, 40
    g = torch.Generator().manual_seed(15)
    X, R, v, u = (torch.randn(M, N, generator=g) for _ in range(4))
    w = torch.rand(N, generator=g) + 0.5
    f32 = torch.float32
    out = dg.rms_norm(padded(X, f32), w.cuda(), residual=padded(R, f32), keep=True, eps=EPS)
    dX, dw = dg.rms_norm_backward(padded(v, f32), out["total"], w.cuda(), out["rstd"], dtotal=padded(u, f32))

    def f(x, ww):
        s, _, y = norm64(x, R, ww)
        return float((v.double() * y).sum() + (u.double() * s).sum())
    h = 1e-5
    for grad, at in ((dX, 0), (dw, 1)):
        d = torch.randn(grad.shape, generator=g).double()
        args = [X.double(), w.double()]
        hi, lo = list(args), list(args)
        hi[at], lo[at] = args[at] + h * d, args[at] - h * d
        ana = grad.cpu().double()
        assert abs(float((ana * d).sum()) - (f(*hi) - f(*lo)) / (2 * h)) <= 1e-5 * float((ana * d).abs().sum()) + 1e-6


def test_backward_in_place_empty_and_without_dweight():
    dY, S = rows(9, 300, torch.bfloat16, 16), rows(9, 300, torch.bfloat16, 17)
    w, rstd = torch.rand(300).cuda(), torch.rand(9).cuda()
    dS = rows(9, 300, torch.bfloat16, 18)
    pad = lambda x: padded(x, torch.bfloat16)  # noqa: E731
    want, _ = dg.rms_norm_backward(pad(dY), pad(S), w, rstd, dtotal=pad(dS))
    a, b = pad(dY), pad(dS)
    dg.rmsnorm_bwd(a, pad(S), w, rstd, a, dtotal=b)
    assert torch.equal(a, want)
    a = pad(dY)
    dg.rmsnorm_bwd(a, pad(S), w, rstd, b, dtotal=b)
    assert torch.equal(b, want)
    e = torch.empty(0, 300, dtype=torch.bfloat16, device="cuda")
    _, dw = dg.rms_norm_backward(e, e, w, torch.empty(0, device="cuda"))
    assert bool((dw == 0).all())


@pytest.mark.parametrize("f8", [False, True])
def test_more_rows_than_a_launch_holds(f8):
    """2^25 + 5 rows of 8 columns (16 lanes each): two launches; the rows behind the
    second one's start are those of a call on them alone."""
    M, N, cut = (1 << 25) + 5, 8, 1 << 25
    X = torch.randn(4096, N, generator=torch.Generator().manual_seed(70)).bfloat16().cuda().repeat(M // 4096 + 1, 1)[:M]
    w = torch.linspace(0.5, 1.5, N, device="cuda")
    out = dg.rms_norm(X, w, residual=X, f8=f8, keep=True, eps=EPS)
    some = dg.rms_norm(X[:4096], w, residual=X[:4096], f8=f8, keep=True, eps=EPS)
    for name, t in out.items():
        t, want = (t.view(torch.uint8), some[name].view(torch.uint8)) if name == "Y" and f8 else (t, some[name])
        for at in (0, cut - 4096):
            assert torch.equal(t[at:at + 4096], want), (name, at)
        assert torch.equal(t[cut:], want[:M - cut]), name
