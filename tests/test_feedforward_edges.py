"""The feed-forward block's operators at the ends of their ranges: sizes of zero under every plan, and rows whose
offsets pass 32 bits."""
import pytest
import torch

import dense_gemm_matrix_amd as dg
from tests.linear_ref import F8, act64, padded

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
PLANS = [None, (16, 32, 1), (32, 32, 1), (64, 64, 1), (128, 128, 1), (128, 128, 3), (256, 256, 1), (256, 256, 2)]


@pytest.fixture(params=PLANS, ids=str)
def plan(request):
    if request.param:
        dg.dgemm_set_plan_override(dg.DGEMM_PLAN_GRID, *request.param)
    yield request.param
    dg.dgemm_set_plan_override(dg.DGEMM_PLAN_AUTO)


def mat(rows, cols, dt, value=1.0):
    """rows x cols in a buffer that has bytes even where there are no columns; NaN past them."""
    return padded(torch.full((rows, cols), value), dt, 1)


def ws(n=1 << 22):
    return torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("fmt", list(DT))
def test_gated_sizes_of_zero(plan, fmt):
    dt = DT[fmt]
    for M in (0, 1, 20, 300):
        for N, K in ((0, 40), (40, 0), (0, 0), (40, 40)):
            if M and N and K:
                continue
            A, Bg, Bu = mat(M, K, dt), mat(K, N, dt), mat(K, N, dt)
            C, G, U = (mat(M, N, dt, float("nan")) for _ in range(3))
            bias = torch.full((N,), 1.5, device="cuda")
            dg.gemm_gated(A, Bg, Bu, C, bias_g=bias, bias_u=bias, act="relu", gate=G, up=U, workspace=ws())
            assert (C == 2.25).all() and (G == 1.5).all() and (U == 1.5).all()
            for want in ("dA dBg dBu", "dA", "dBg", "dBu"):
                outs = {k: mat(*s, dt, float("nan")) for k, s in
                        (("dA", (M, K)), ("dBg", (K, N)), ("dBu", (K, N))) if k in want.split()}
                sums = {k: torch.full((N,), float("nan"), device="cuda") for k in ("dbias_g", "dbias_u")}
                g = mat(M, N, dt)
                dg.gemm_gated_bwd(A, Bg, Bu, g, g, g, act="none", workspace=ws(), **outs, **sums)
                assert all((t == 0).all() for t in outs.values())
                assert all((t == M).all() for t in sums.values())


@pytest.mark.parametrize("od", list(DT.values()), ids=str)
@pytest.mark.parametrize("rows_b", [1, 128])
def test_8_bit_sizes_of_zero(plan, od, rows_b):
    for M in (0, 1, 20, 300):
        for N, K in ((0, 40), (40, 0), (0, 0), (40, 40)):
            if M and N and K:
                continue
            kb, nb = (K + 127) // 128, N if rows_b == 1 else (N + 127) // 128
            C = mat(M, N, od, float("nan"))
            dg.gemm_f8_block(mat(M, K, F8), mat(N, K, F8), C, torch.ones(M, kb, device="cuda"),
                             torch.ones(nb, kb, device="cuda"), bias=torch.full((N,), 1.5, device="cuda"),
                             residual=mat(M, N, od), workspace=ws())
            assert (C == 2.5).all()


def ints(rows, cols, dt, seed):
    """Values -1, 0 and 1, whose sums are exact whatever their order."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-1, 2, (rows, cols), generator=g, device="cuda", dtype=torch.int8).to(dt)


def parts(M, n=300):
    """The first rows, rows around element 2^31 / 8192 and the last."""
    return [slice(0, n), slice(262144 - n, 262144 + n), slice(M - n, M)]


def test_gated_rows_past_32_bits():
    """A and dA of 2.2e9 values: every row is where it belongs, and every row counts in the weights' gradients."""
    M, N, K, dt = 270_001, 40, 8192, torch.bfloat16
    A, Bg, Bu = ints(M, K, dt, 1), ints(K, N, dt, 2), ints(K, N, dt, 3)
    C, G, U = dg.linear_gated(A, Bg, Bu, act="relu", keep_preact=True, out_dtype=torch.float32)
    for r in parts(M):
        a = A[r].float().cpu()
        g, u = a @ Bg.float().cpu(), a @ Bu.float().cpu()
        assert torch.equal(G[r].cpu(), g) and torch.equal(U[r].cpu(), u)
        assert torch.equal(C[r].cpu(), act64(g.double(), "relu").float() * u)
    del C, G, U
    dC, G, U = ints(M, N, dt, 4), ints(M, N, dt, 5), ints(M, N, dt, 6)
    dA, dBg, dBu, dbg, dbu = dg.linear_gated_backward(A, Bg, Bu, dC, G, U, act="none", bias=True)
    dg_, du = (dC.float() * U.float()), (dC.float() * G.float())
    assert torch.equal(dbg, dg_.sum(0)) and torch.equal(dbu, du.sum(0))
    for r in parts(M):
        want = dg_[r].cpu() @ Bg.float().t().cpu() + du[r].cpu() @ Bu.float().t().cpu()
        assert torch.equal(dA[r].float().cpu(), want.to(dt).float())
    for got, d in ((dBg, dg_), (dBu, du)):
        want = torch.zeros(K, N, dtype=torch.float64, device="cuda")
        for r in range(0, M, 30_000):
            want += torch.mm(A[r:r + 30_000].double().t().contiguous(), d[r:r + 30_000].double())
        assert torch.equal(got, want.to(dt))


def test_8_bit_rows_past_32_bits():
    """A quantizer's rows, its transposed columns and a product's rows past 2^31 bytes and values."""
    M, N, K, dt = 270_001, 40, 8192, torch.bfloat16
    X = ints(M, K, dt, 1)
    X[::3, 5] = 3.5
    Q, s = dg.quantize_f8_block(X)
    B = ints(N, K, F8, 2)
    sb = torch.ones(1, K // 128, device="cuda")
    C = dg.matmul_f8_block(Q, B, s, sb, out_dtype=torch.float32)
    for r in parts(M):
        few, sf = dg.quantize_f8_block(X[r].clone())
        assert torch.equal(Q[r].view(torch.uint8), few.view(torch.uint8)) and torch.equal(s[r], sf)
        want = (few.double() * sf.double().repeat_interleave(128, 1)).cpu() @ B.double().t().cpu()
        # the scales' quotients by 448 are off by half a step each
        assert torch.allclose(C[r].cpu().double(), want, rtol=0, atol=K * 2.0 ** -22)
    del C, Q, s
    T, st = dg.quantize_f8_block(X, transpose=True)
    W, sw = dg.quantize_f8_block(X, rows=128)
    for r in (slice(0, 256), slice(262144 - 128, 262144 + 128), slice(M // 128 * 128 - 128, M)):
        few, sf = dg.quantize_f8_block(X[r].clone(), transpose=True)
        assert torch.equal(T[:, r].contiguous().view(torch.uint8), few.contiguous().view(torch.uint8))
        assert torch.equal(st[:, r.start // 128:(r.stop + 127) // 128], sf)
        few, sf = dg.quantize_f8_block(X[r].clone(), rows=128)
        assert torch.equal(W[r].view(torch.uint8), few.view(torch.uint8))
        assert torch.equal(sw[r.start // 128:(r.stop + 127) // 128], sf)


@pytest.mark.parametrize("f8", [False, "row", "block"])
def test_layer_norm_rows_past_32_bits(f8):
    """Bit for bit the rows of a call on them alone (of more than 256 rows, as few have another order of sums)."""
    M, N, dt = 270_001, 8192, torch.bfloat16
    X = ints(M, N, dt, 1)
    w, b = torch.rand(N, device="cuda") + 0.5, torch.randn(N, device="cuda")
    out = dg.layer_norm(X, w, b, f8=f8, keep=True)
    for r in parts(M):
        few = dg.layer_norm(X[r].clone(), w, b, f8=f8, keep=True)
        for k in few:
            got = out[k][r]
            same = torch.equal(got.view(torch.uint8), few[k].view(torch.uint8)) if got.dtype == F8 else \
                torch.equal(got, few[k])
            assert same, k
    if f8:
        return
    dY = ints(M, N, dt, 2)
    dX, dw, db = dg.layer_norm_backward(dY, X, w, out["mean"], out["rstd"])
    assert torch.equal(db, dY.sum(0, dtype=torch.float32))
    for r in parts(M):
        few = dg.layer_norm_backward(dY[r].clone(), X[r].clone(), w, out["mean"][r].clone(), out["rstd"][r].clone())
        assert torch.equal(dX[r], few[0])
    xh = torch.zeros(N, dtype=torch.float64, device="cuda")
    size = torch.zeros(N, dtype=torch.float64, device="cuda")
    for r in range(0, M, 30_000):
        q = slice(r, r + 30_000)
        t = dY[q].double() * (X[q].double() - out["mean"][q].double()[:, None]) * out["rstd"][q].double()[:, None]
        xh += t.sum(0)
        size += t.abs().sum(0)
    assert ((dw.double() - xh).abs() <= (M + 5) * 2.0 ** -24 * size).all()
