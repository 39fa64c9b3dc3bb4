"""gemm_act, gemm_act_bwd and gemm_f8 on the GPU against plain 64-bit forms."""
import ctypes
import threading

import pytest
import torch

import dense_gemm_matrix_amd as dg
from tests.linear_ref import (F8, SLOPE, TINY, U, act64, act_grad64, gap_kept, linear64, out_bound, padded,
                              quant64, sentinel, sum_bound, within)

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "f32x3": torch.float32}


@pytest.fixture
def grid_plan():
    """Forces a tile and split count for the test."""
    def force(rows, cols, splits=1):
        dg.dgemm_set_plan_override(dg.DGEMM_PLAN_GRID, rows, cols, splits)
    yield force
    dg.dgemm_set_plan_override(dg.DGEMM_PLAN_AUTO)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def inputs(M, N, K, dt, seed, bias=True, residual=True, out=None):
    g = gen(seed)
    A = torch.randn(M, K, generator=g).to(dt)
    B = (torch.randn(K, N, generator=g) / max(1, K) ** 0.5).to(dt)
    b = torch.randn(N, generator=g) if bias else None
    R = torch.randn(M, N, generator=g).to(out or dt) if residual else None
    return A, B, b, R


def run_act(fmt, out, M, N, K, act, seed=0, bias=True, residual=True, preact=True, ws_bytes=0, extra=1):
    dt = DT[fmt]
    od = torch.float32 if out == "f32" else dt
    A, B, b, R = inputs(M, N, K, dt, seed, bias, residual, od)
    Ad, Bd = padded(A, dt, extra), padded(B, dt, extra)
    Rd = None if R is None else padded(R, od, 2 * extra)
    C = sentinel(M, N, od)
    Z = sentinel(M, N, od, 2) if preact else None
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device="cuda") if ws_bytes else None
    dg.gemm_act(Ad, Bd, C, bias=None if b is None else b.cuda(), act=act, residual=Rd, preact=Z, workspace=ws,
                in_fmt=fmt)
    torch.cuda.synchronize()
    C64, Z64, S = linear64(A, B, b, act, R)
    dz = sum_bound(K, S, fmt == "f32x3")
    within(C, C64, out_bound(C64, Z64, dz, R, od, act))
    assert gap_kept(C)
    if preact:
        within(Z, Z64, dz + U[od] * (Z64.abs() + dz) + TINY[od])
        assert gap_kept(Z)


# Sizes: few rows (the register-streaming kernel), one slice-K tile and more,
# odd everything, one column, and K of 1, below, at and above a step.
SHAPES = [(1, 1, 1), (1, 33, 40), (1, 200, 515), (2, 40, 9000), (5, 130, 33), (16, 97, 257), (17, 70, 65), (33, 8, 130),
          (70, 129, 200), (130, 300, 72)]


@pytest.mark.parametrize("fmt, out", [("bf16", "same"), ("bf16", "f32"), ("f16", "same"), ("f16", "f32"),
                                      ("f32", "f32"), ("f32x3", "f32")])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward(fmt, out, shape):
    acts = list(dg.ACT_CODES)
    i = SHAPES.index(shape)
    run_act(fmt, out, *shape, acts[i % 5], seed=i)
    run_act(fmt, out, *shape, acts[(i + 2) % 5], seed=i + 50, bias=i % 2 == 0, residual=i % 3 == 0, preact=False)


@pytest.mark.parametrize("act", list(dg.ACT_CODES))
@pytest.mark.parametrize("fmt", ["bf16", "f16", "f32"])
def test_every_activation(act, fmt):
    run_act(fmt, "same", 40, 72, 96, act, seed=3)
    run_act(fmt, "same", 3, 72, 96, act, seed=4)


# The grid tiles with ragged edges, forced, unsplit and split.
@pytest.mark.parametrize("fmt, tile", [("bf16", (256, 256)), ("bf16", (192, 256)), ("bf16", (128, 128)),
                                       ("f16", (256, 256)), ("f16", (128, 128)), ("f32", (128, 128)),
                                       ("f32x3", (256, 256)), ("f32x3", (128, 128))])
@pytest.mark.parametrize("splits", [1, 3])
def test_forward_grid_tiles(grid_plan, fmt, tile, splits):
    grid_plan(*tile, splits)
    ws = 0 if splits == 1 else 8 << 20
    run_act(fmt, "same", 300, 270, 200, "gelu_tanh", seed=11, ws_bytes=ws)
    run_act(fmt, "same", 261, 515, 328, "silu", seed=12, bias=False, ws_bytes=ws)
    run_act(fmt, "f32", 130, 31, 64, "gelu", seed=13, residual=False, ws_bytes=ws)


@pytest.mark.parametrize("cols", [32, 64, 128])
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("fmt", ["bf16", "f16", "f32"])
def test_forward_few_row_strips(grid_plan, cols, splits, fmt):
    grid_plan(16, cols, splits)
    ws = 0 if splits == 1 else 1 << 20
    for i, (M, N, K) in enumerate([(1, 300, 1030), (16, 129, 64), (7, 20, 333)]):
        run_act(fmt, "same", M, N, K, "silu", seed=20 + i, ws_bytes=ws)
        run_act(fmt, "f32", M, N, K, "none", seed=30 + i, ws_bytes=ws, preact=False)


@pytest.mark.parametrize("fmt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", [(1, 4100, 4096), (16, 2050, 4130), (5, 130, 8200), (3, 70, 16500)],
                         ids=lambda s: "x".join(map(str, s)))
def test_forward_few_rows_deep(fmt, shape):
    """The planner's own splits of few-row products, K a multiple of their step and not."""
    assert dg.gemm_act_plan(fmt, *shape, 1 << 24, fmt != "f32")["splits"] > 1
    run_act(fmt, "same", *shape, "silu", seed=20, ws_bytes=1 << 24)


def test_integers_are_exact():
    """Small integers: every sum is exact, so the output is its one rounding."""
    for M, N, K in [(1, 70, 100), (16, 40, 64), (40, 72, 96), (300, 264, 200)]:
        g = gen(M)
        A = torch.randint(-8, 9, (M, K), generator=g).double()
        B = torch.randint(-8, 9, (K, N), generator=g).double()
        b = torch.randint(-8, 9, (N,), generator=g).float()
        R = torch.randint(-8, 9, (M, N), generator=g).double()
        for fmt, dt in (("bf16", torch.bfloat16), ("f16", torch.float16), ("f32", torch.float32)):
            C = sentinel(M, N, dt)
            dg.gemm_act(padded(A, dt), padded(B, dt), C, bias=b.cuda(), act="relu", residual=padded(R, dt))
            assert torch.equal(C.cpu(), ((A @ B + b.double()).clamp_min(0) + R).to(dt))


def test_residual_in_place_and_column_window():
    """residual may be C itself; a window of a wider buffer keeps its surroundings."""
    for M, N, K in [(3, 40, 64), (50, 40, 64), (300, 264, 72)]:
        A, B, b, R = inputs(M, N, K, torch.bfloat16, 5)
        want = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        pad = lambda x: padded(x, torch.bfloat16)  # noqa: E731
        Rd = pad(R)
        wide = torch.full((M, N + 64), 7.0, dtype=torch.bfloat16, device="cuda")
        C = wide[:, 16:16 + N]
        C.copy_(R)
        dg.gemm_act(pad(A), pad(B), want, bias=b.cuda(), act="gelu", residual=Rd)
        dg.gemm_act(pad(A), pad(B), C, bias=b.cuda(), act="gelu", residual=C)
        assert torch.equal(C, want)
        assert bool((wide[:, :16] == 7).all()) and bool((wide[:, 16 + N:] == 7).all())


@pytest.mark.parametrize("tile, splits", [((256, 256), 1), ((128, 128), 1), ((128, 128), 3), ((64, 64), 4),
                                          ((32, 32), 8)])
def test_residual_in_place_in_every_plan(grid_plan, tile, splits):
    """C := act(..) + C where the residual is C itself, in the 16-bit and 8-bit products."""
    grid_plan(*tile, splits)
    M, N, K = 290, 270, 200
    A, B, b, R = inputs(M, N, K, torch.bfloat16, 15)
    pad = lambda x: padded(x, torch.bfloat16)  # noqa: E731
    Rd = pad(R)
    ws = torch.empty(4 << 20, dtype=torch.uint8, device="cuda")
    want, C = sentinel(M, N, torch.bfloat16), pad(R)
    dg.gemm_act(pad(A), pad(B), want, bias=b.cuda(), act="silu", residual=Rd, workspace=ws)
    dg.gemm_act(pad(A), pad(B), C, bias=b.cuda(), act="silu", residual=C, workspace=ws)
    assert torch.equal(C, want)
    A8, B8, sa, sb, _, _ = f8_inputs(M, N, K, 16)
    A8, B8, sa, sb = padded(A8, F8), padded(B8, F8), sa.cuda(), sb.cuda()
    want, C = sentinel(M, N, torch.bfloat16), pad(R)
    dg.gemm_f8(A8, B8, want, sa, sb, act="gelu", residual=Rd, workspace=ws)
    dg.gemm_f8(A8, B8, C, sa, sb, act="gelu", residual=C, workspace=ws)
    assert torch.equal(C, want)


def test_empty_sums_and_sizes():
    b = torch.randn(40, generator=gen(1))
    for M in (1, 20, 300):
        A = torch.empty(M, 0, dtype=torch.bfloat16, device="cuda")
        B = torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")
        C = sentinel(M, 40, torch.bfloat16)
        dg.gemm_act(A, B, C, bias=b.cuda(), act="relu")
        assert torch.equal(C.cpu(), b.clamp_min(0).to(torch.bfloat16).expand(M, 40))
    C = torch.empty(0, 40, dtype=torch.bfloat16, device="cuda")
    dg.gemm_act(torch.empty(0, 8, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(8, 40, dtype=torch.bfloat16, device="cuda"), C, act="silu")


@pytest.mark.parametrize("fmt", ["bf16", "f32"])
@pytest.mark.parametrize("M", [4, 40])
def test_nonfinite_values_stay_in_their_rows_and_columns(fmt, M):
    N, K = 72, 70
    dt = DT[fmt]
    A, B, b, R = inputs(M, N, K, dt, 6)
    A[2, 5] = float("nan")
    B[3, 7] = float("inf")
    R[1, 9] = float("nan")
    R[0, 10] = float("-inf")
    C = sentinel(M, N, dt)
    dg.gemm_act(padded(A, dt), padded(B, dt), C, bias=b.cuda(), act="relu", residual=padded(R, dt))
    C = C.cpu().float()
    assert torch.isnan(C[2]).all() and torch.isnan(C[1, 9]) and C[0, 10] == float("-inf")
    # relu of +-infinity: infinity or 0 by the sign of A's element
    for i in range(M):
        if i != 2:
            assert C[i, 7] == float("inf") or A[i, 3] <= 0
    ok = torch.ones(M, N, dtype=torch.bool)
    ok[2], ok[:, 7], ok[1, 9], ok[0, 10] = False, False, False, False
    assert torch.isfinite(C[ok]).all()


def test_large_preactivations_saturate():
    """Far out the activations are the identity or zero, without NaN."""
    for fmt in ("bf16", "f32"):
        dt = DT[fmt]
        z = torch.tensor([[-3e38, -1e20, -1e4, -200.0, -40.0, 0.0, 40.0, 200.0, 1e4, 1e20, 3e38]]).to(dt)
        one = torch.ones(1, 1, dtype=dt)
        want = torch.where(z > 0, z, torch.zeros_like(z)).float()
        for act in ("gelu", "gelu_tanh", "silu"):
            for rows in (1, 20):
                C = sentinel(rows, 11, dt)
                dg.gemm_act(padded(one.expand(rows, 1), dt), padded(z, dt), C, act=act)
                got = C.cpu().float()
                assert torch.allclose(got, want.expand(rows, 11), rtol=1e-2, atol=1e-12), (fmt, act, got[0])


# ------------------------------------------------------------------- backward

def bwd64(A, B, dC, Z, act, dz_dtype):
    """(dA, dB, dbias) in 64 bits, their absolute sums, and the error bound of dZ:
    the derivative in fp32 within 64 half steps of 1 + |z| times |dC| (some dozen
    operations on values of at most a few times that), and its rounding."""
    dC, A, B = dC.double(), A.double(), B.double()
    dZ = dC if act == "none" else dC * act_grad64(Z.double(), act)
    e = torch.zeros_like(dZ) if act == "none" else 64 * 2.0 ** -24 * dC.abs() * (1 + Z.double().abs())
    r = e + U[dz_dtype] * (dZ.abs() + e) + TINY[dz_dtype]
    return dZ, e, r, A, B


def run_bwd(fmt, out, M, N, K, act, seed, ws=None, want=("dA", "dB", "dbias")):
    dt = DT[fmt]
    cd = torch.float32 if out == "f32" else dt
    g = gen(seed)
    A = torch.randn(M, K, generator=g).to(dt)
    B = (torch.randn(K, N, generator=g) / max(1, K) ** 0.5).to(dt)
    dC = torch.randn(M, N, generator=g).to(cd)
    Z = torch.randn(M, N, generator=g).to(cd) if act != "none" else None
    dA = sentinel(M, K, dt) if "dA" in want else None
    dB = sentinel(K, N, dt) if "dB" in want else None
    db = torch.full((N,), float("nan"), device="cuda") if "dbias" in want else None
    req, best = dg.gemm_act_bwd_workspace(fmt, M, N, K, act, cd == dt and fmt[:3] != "f32")
    n = {None: best, "least": req}[ws]
    work = torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda")
    dg.gemm_act_bwd(padded(A, dt, 1), padded(B, dt, 1), padded(dC, cd, 1), dA=dA, dB=dB, dbias=db,
                    preact=None if Z is None else padded(Z, cd, 2), act=act, workspace=work, in_fmt=fmt)
    torch.cuda.synchronize()
    dZ, e, r, A, B = bwd64(A, B, dC, Z, act, dt if (act != "none" or cd != dt) else torch.float64)
    if act == "none" and cd == dt:
        r = torch.zeros_like(dZ)
    x3 = fmt == "f32x3"
    if dA is not None:
        ref = dZ @ B.t()
        b = (r @ B.abs().t()) + sum_bound(N, (dZ.abs() + r) @ B.abs().t(), x3)
        within(dA, ref, b + U[dt] * (ref.abs() + b) + TINY[dt])
        assert gap_kept(dA)
    if dB is not None:
        ref = A.t() @ dZ
        b = (A.abs().t() @ r) + sum_bound(M, A.abs().t() @ (dZ.abs() + r), x3)
        within(dB, ref, b + U[dt] * (ref.abs() + b) + TINY[dt])
        assert gap_kept(dB)
    if db is not None:
        within(db, dZ.sum(0), e.sum(0) + (M + 2) * 2.0 ** -24 * (dZ.abs() + e).sum(0) + 2.0 ** -149)


U[torch.float64], TINY[torch.float64] = 0.0, 0.0


@pytest.mark.parametrize("fmt, out", [("bf16", "same"), ("bf16", "f32"), ("f16", "same"), ("f16", "f32"),
                                      ("f32", "f32"), ("f32x3", "f32")])
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 130, 72), (3, 40, 33), (64, 64, 64), (65, 200, 129),
                                   (300, 270, 140), (513, 40, 24)], ids=lambda s: "x".join(map(str, s)))
def test_backward(fmt, out, shape):
    acts = list(dg.ACT_CODES)
    i = sum(shape)
    run_bwd(fmt, out, *shape, acts[i % 5], seed=i)
    run_bwd(fmt, out, *shape, acts[(i + 1) % 5], seed=i + 1, ws="least")


@pytest.mark.parametrize("act", list(dg.ACT_CODES))
@pytest.mark.parametrize("fmt", ["bf16", "f32"])
def test_backward_every_activation(act, fmt):
    run_bwd(fmt, "same", 70, 136, 90, act, seed=7)


@pytest.mark.parametrize("tile, splits", [((256, 256), 1), ((128, 128), 1), ((256, 256), 2), ((128, 128), 3)])
@pytest.mark.parametrize("fmt", ["bf16", "f16"])
def test_backward_grid_tiles(grid_plan, tile, splits, fmt):
    grid_plan(*tile, splits)
    run_bwd(fmt, "same", 300, 270, 261, "silu", seed=8)
    run_bwd(fmt, "same", 520, 136, 390, "none", seed=9)
    for want in (("dA",), ("dB",), ("dB", "dbias")):
        run_bwd(fmt, "same", 390, 300, 136, "silu", seed=10, want=want)


@pytest.mark.parametrize("tile, waves", [(32, 4), (32, 8), (64, 4)])
@pytest.mark.parametrize("fmt", ["bf16", "f16"])
def test_backward_slice_tiles(grid_plan, tile, waves, fmt):
    """The slice-K tiles, runs of blocks from none to several per wave, K tails."""
    grid_plan(tile, tile, waves)
    for i, (M, N, K) in enumerate([(17, 40, 33), (70, 136, 90), (130, 72, 261), (1000, 65, 70), (40, 1100, 24)]):
        run_bwd(fmt, "same", M, N, K, "silu", seed=40 + i)
        run_bwd(fmt, "same", M, N, K, "none", seed=50 + i)


@pytest.mark.parametrize("fmt", ["bf16", "f16", "f32", "f32x3"])
@pytest.mark.parametrize("shape", [(50, 30, 20), (400, 70, 500), (90, 700, 150), (917, 415, 1035), (240, 1501, 430),
                                   (2000, 300, 200), (33, 2000, 1000),
                                   (600, 801, 1500), (1030, 1100, 520)], ids=lambda s: "x".join(map(str, s)))
def test_backward_products_together(fmt, shape):
    """Layers whose products share a launch: small tiles in both orders, with fewer
    and more workgroups than CUs, and grid tiles."""
    run_bwd(fmt, "same", *shape, "silu", seed=60)
    run_bwd(fmt, "f32", *shape, "none", seed=61, want=("dA", "dB"))
    run_bwd(fmt, "same", *shape, "relu", seed=62, want=("dB", "dbias"))


@pytest.mark.parametrize("want", [("dA",), ("dB",), ("dbias",), ("dA", "dbias"), ("dB", "dbias"), ("dA", "dB")])
def test_backward_parts(want):
    for act in ("none", "gelu"):
        run_bwd("bf16", "same", 70, 136, 90, act, seed=10, want=want)
        run_bwd("f32", "f32", 70, 36, 90, act, seed=10, want=want)


@pytest.mark.parametrize("N", [1, 8, 64, 65, 128, 130, 256, 257, 513, 1100])
@pytest.mark.parametrize("M", [17, 64, 65, 131, 1003])
def test_backward_widths(M, N):
    """Several rows per wave of narrow layers, whole and part passes, one and many
    workgroups per column block."""
    run_bwd("bf16", "same", M, N, 24, "silu", seed=M + N)
    run_bwd("bf16", "f32", M, N, 24, "gelu", seed=M + N + 1, want=("dbias",))


def test_backward_against_differences():
    """The gradient of sum(w o C) by central differences of the plain 64-bit
    forward, along random directions.  The fp32 kernel's own error is within
    1e-5 of the gradient's size here (K, M, N of a few dozen: 40 half steps of
    sums), the differences' within h^2 times third derivatives and 2^-52 / h."""
    M, N, K = 24, 20, 28
    g = gen(12)
    A, B, b, _ = inputs(M, N, K, torch.float32, 12)
    w = torch.randn(M, N, generator=g)
    for act in ("gelu", "gelu_tanh", "silu"):
        A64, B64, b64 = A.double(), B.double(), b.double()
        C, Z = dg.linear(padded(A, torch.float32), padded(B, torch.float32), bias=b.cuda(), act=act,
                         keep_preact=True)
        dA, dB, db = dg.linear_backward(padded(A, torch.float32), padded(B, torch.float32),
                                        padded(w, torch.float32), preact=Z, act=act, bias=True)
        f = lambda a, bb, c: float((w.double() * act64(a @ bb + c, act)).sum())  # noqa: E731
        h = 1e-5
        for grad, at in ((dA, 0), (dB, 1), (db, 2)):
            d = torch.randn(grad.shape, generator=g).double()
            args = [A64, B64, b64]
            hi, lo = list(args), list(args)
            hi[at], lo[at] = args[at] + h * d, args[at] - h * d
            num = (f(*hi) - f(*lo)) / (2 * h)
            ana = grad.cpu().double()
            assert abs(float((ana * d).sum()) - num) <= 1e-5 * float((ana.abs() * d.abs()).sum()) + 1e-6


def test_backward_empty_sums():
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    dA, dB, db = dg.linear_backward(z(0, 8), z(8, 16), z(0, 16), bias=True)
    assert dA.shape == (0, 8) and bool((dB == 0).all()) and bool((db == 0).all())
    for M in (4, 40, 300):
        dA, dB, _ = dg.linear_backward(z(M, 8), z(8, 0), z(M, 0))
        assert bool((dA == 0).all()) and dB.shape == (8, 0)
        dA, dB, db = dg.linear_backward(z(M, 0), z(0, 16), z(M, 16) + 1, bias=True)
        assert dA.shape == (M, 0) and dB.shape == (0, 16) and bool((db == M).all())


# ---------------------------------------------------------------- 8-bit product

def f8_inputs(M, N, K, seed):
    g = gen(seed)
    q = lambda r, c: torch.randn(r, c, generator=g).mul(8).to(F8)  # noqa: E731
    return (q(M, K), q(N, K), torch.rand(M, generator=g) * 0.1 + 0.01, torch.rand(N, generator=g) * 0.1 + 0.01,
            torch.randn(N, generator=g), torch.randn(M, N, generator=g))


def run_f8(M, N, K, od, act, seed, bias=True, residual=True, ws_bytes=0):
    A, B, sa, sb, b, R = f8_inputs(M, N, K, seed)
    R = R.to(od) if residual else None
    C = sentinel(M, N, od)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device="cuda") if ws_bytes else None
    dg.gemm_f8(padded(A, F8, 1), padded(B, F8, 2), C, sa.cuda(), sb.cuda(), bias=b.cuda() if bias else None,
               act=act, residual=None if R is None else padded(R, od, 1), workspace=ws)
    torch.cuda.synchronize()
    s = sa.double()[:, None] * sb.double()
    Z = (A.double() @ B.double().t()) * s
    S = (A.double().abs() @ B.double().abs().t()) * s
    if bias:
        Z, S = Z + b.double(), S + b.double().abs()
    C64 = act64(Z, act)
    C64 = C64 if R is None else C64 + R.double()
    dz = sum_bound(K + 2, S)
    if od != torch.float32 and M > 16:
        # the 8-bit instruction drops, of each product, what lies below 2^-13 of
        # the largest near it: at most 2^-13 of the largest product for each k
        dz = dz + K * 2.0 ** -13 * s * (A.double().abs().amax(1)[:, None] * B.double().abs().amax(1))
    within(C, C64, out_bound(C64, Z, dz, R, od, act))
    assert gap_kept(C)


F8_SHAPES = [(1, 1, 1), (1, 130, 300), (16, 33, 129), (5, 16, 1024), (17, 40, 100), (64, 64, 64),
             (130, 300, 257), (257, 270, 515)]


@pytest.mark.parametrize("od", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape", F8_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_f8(od, shape):
    acts = list(dg.ACT_CODES)
    i = F8_SHAPES.index(shape)
    run_f8(*shape, od, acts[i % 5], seed=i)
    run_f8(*shape, od, acts[(i + 3) % 5], seed=i, bias=i % 2 == 0, residual=i % 2 == 1)


@pytest.mark.parametrize("shape", [(3, 4109, 40), (16, 4200, 2050), (1, 4100, 5000)],
                         ids=lambda s: "x".join(map(str, s)))
def test_few_rows_of_wide_outputs(shape):
    """More strips than CUs: fewer waves each, short and long K; the same strips for
    the 16-bit and fp32 gradients of A."""
    M, N, K = shape
    run_f8(M, N, K, torch.bfloat16, "silu", seed=31)
    run_f8(M, N, K, torch.float32, "none", seed=32)
    run_bwd("bf16", "same", M, K, N, "silu", seed=33, want=("dA",))
    run_bwd("f32", "f32", M, K, N, "silu", seed=34, want=("dA",))


@pytest.mark.parametrize("tile, splits", [((256, 256), 1), ((128, 128), 1), ((256, 256), 2), ((128, 128), 3)])
def test_f8_grid_tiles(grid_plan, tile, splits):
    grid_plan(*tile, splits)
    for i, (M, N, K) in enumerate([(300, 270, 400), (129, 515, 1000), (64, 31, 272)]):
        run_f8(M, N, K, torch.bfloat16, "silu", seed=i, ws_bytes=4 << 20)
        run_f8(M, N, K, torch.float32, "none", seed=i, ws_bytes=4 << 20)


@pytest.mark.parametrize("tile, waves", [(32, 4), (32, 8), (64, 4)])
def test_f8_slice_tiles(grid_plan, tile, waves):
    grid_plan(tile, tile, waves)
    for i, (M, N, K) in enumerate([(17, 40, 100), (64, 31, 272), (70, 100, 1025), (130, 72, 2300)]):
        for od in (torch.float32, torch.bfloat16, torch.float16):
            run_f8(M, N, K, od, "silu", seed=i)


def test_f8_every_value():
    """Every finite e4m3 code times 1 in each position of a 128-k step."""
    codes = torch.arange(256, dtype=torch.uint8)
    codes = codes[(codes & 0x7f) != 0x7f]
    v = codes.view(F8)
    for M in (2, 40, 1100):  # the few-row kernel, a slice-K tile, a grid tile
        B_rows = len(v) if M < 1000 else 1024
        for k in (0, 31, 32, 63, 64, 100, 127, 128):
            A = torch.zeros(M, 129, dtype=F8)
            A[:, k] = torch.ones(M).to(F8)
            B = torch.zeros(B_rows, 129, dtype=F8)
            B[:len(v), k] = v
            for od in (torch.float32, torch.bfloat16):
                C = dg.matmul_f8(padded(A, F8), padded(B, F8), torch.ones(M).cuda(),
                                 torch.ones(B_rows).cuda(), out_dtype=od)
                assert torch.equal(C[:, :len(v)].cpu().float(), v.float().expand(M, len(v)))


def test_f8_row_scales_of_nan_fill_their_rows():
    A, B, sa, sb, b, R = f8_inputs(20, 40, 64, 3)
    sa[3] = float("nan")
    C = dg.matmul_f8(padded(A, F8), padded(B, F8), sa.cuda(), sb.cuda()).float().cpu()
    assert torch.isnan(C[3]).all() and torch.isfinite(C[:3]).all() and torch.isfinite(C[4:]).all()


# ------------------------------------------------------ streams, graphs, threads

def calls(seed):
    """A serving block and a training step on small shapes: a function that runs
    them into fixed buffers, and the buffers."""
    M, N, K = 40, 136, 96
    g = gen(seed)
    bf = torch.bfloat16
    X, W = torch.randn(M, K, generator=g), torch.randn(K, N, generator=g) / 10
    V_, R = torch.randn(N, K, generator=g) / 10, torch.randn(M, K, generator=g)
    X, W, V_, R = (padded(t, bf) for t in (X, W, V_, R))
    nw = torch.rand(K, generator=g).cuda() + 0.5
    bias = torch.randn(N, generator=g).cuda()
    W8, sw = dg.quantize_f8(W, transpose=True)
    V8, sv = dg.quantize_f8(V_, transpose=True)
    S, Y = sentinel(M, K, bf), sentinel(M, K, F8)
    sy, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    H, H8, sh = sentinel(M, N, bf), sentinel(M, N, F8), torch.empty(M, device="cuda")
    O = sentinel(M, K, bf)
    Yn, Z, T, dT, dH, dYn, dX = (sentinel(M, c, bf) for c in (K, N, N, N, N, K, K))
    dW, dV, db, dnw = sentinel(K, N, bf), sentinel(N, K, bf), torch.empty(N, device="cuda"), torch.empty(K, device="cuda")
    O2 = sentinel(M, K, bf)
    ws = torch.empty(4 << 20, dtype=torch.uint8, device="cuda")

    def run():
        dg.rmsnorm(X, nw, Y, residual=R, total=S, scale=sy)
        dg.gemm_f8(Y, W8, H, sy, sw, bias=bias, act="silu", workspace=ws)
        dg.quant_f8(H, H8, sh)
        dg.gemm_f8(H8, V8, O, sh, sv, residual=S, workspace=ws)
        dg.rmsnorm(X, nw, Yn, residual=R, total=S, rstd=rstd)
        dg.gemm_act(Yn, W, T, bias=bias, act="gelu_tanh", preact=Z, workspace=ws)
        dg.gemm_act(T, V_, O2, residual=S, workspace=ws)
        dg.gemm_act_bwd(T, V_, R, dA=dH, dB=dV, workspace=ws)
        dg.gemm_act_bwd(Yn, W, dH, dA=dYn, dB=dW, dbias=db, preact=Z, act="gelu_tanh", workspace=ws)
        dg.rmsnorm_bwd(dYn, S, nw, rstd, dX, dtotal=R, dweight=dnw, workspace=ws)
    outs = [S, Y, sy, H, H8, sh, O, Yn, rstd, Z, T, O2, dH, dV, dYn, dW, db, dX, dnw]
    data = dict(X=X, W=W, V=V_, R=R, nw=nw, bias=bias, S=S, O2=O2, dX=dX, dW=dW, dV=dV, db=db, dnw=dnw, O=O)
    return run, outs, data


def bits(outs):
    return [o.clone().contiguous().view(torch.uint8).cpu() for o in outs]


def test_block_against_64_bits():
    """Norm, product, activation, product with residual, and the way back, against
    autograd in 64 bits.  bf16 rounds each stored tensor by 2^-8 of its size; a
    result passes at most 8 of them, each adding to the 2-norm at most in full."""
    run, outs, d = calls(1)
    run()
    torch.cuda.synchronize()
    X, W, V_, R = (d[k].cpu().double().requires_grad_(k != "R") for k in "XWVR")
    nw, bias = d["nw"].cpu().double().requires_grad_(True), d["bias"].cpu().double().requires_grad_(True)
    S = X + R
    Y = S * (S.square().mean(1, keepdim=True) + 1e-6).rsqrt() * nw
    O = torch.nn.functional.gelu(Y @ W + bias, approximate="tanh") @ V_ + S
    gX, gW, gV, gn, gb = torch.autograd.grad((O * R).sum(), (X, W, V_, nw, bias))
    tol = 8 * 2.0 ** -8
    for got, ref in ((d["O2"], O), (d["dX"], gX), (d["dW"], gW), (d["dV"], gV), (d["dnw"], gn), (d["db"], gb)):
        ref = ref.detach()
        assert float((got.cpu().double() - ref).norm() / ref.norm()) <= tol
    # in 8 bits two operands of each product are rounded by 2^-4 of their values
    H = (torch.nn.functional.silu(Y @ W + bias) @ V_ + S).detach()
    assert float((d["O"].cpu().double() - H).norm() / H.norm()) <= 4 * 2.0 ** -4


def test_captured_graph_replays():
    run, outs, d = calls(2)
    run()
    torch.cuda.synchronize()
    want = bits(outs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            run()
    torch.cuda.synchronize()
    for i in range(3):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(bits(outs), want)), i
        run()
        torch.cuda.synchronize()


def test_results_are_the_same_every_time_and_on_another_stream():
    run, outs, _ = calls(3)
    run()
    torch.cuda.synchronize()
    want = bits(outs)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(bits(outs), want))


def test_stream_argument_and_threads():
    """The allocating forms on streams of their own, from several threads."""
    A, B, b, R = inputs(33, 72, 100, torch.bfloat16, 4)
    Ad, Bd, Rd, bd = padded(A, torch.bfloat16), padded(B, torch.bfloat16), padded(R, torch.bfloat16), b.cuda()
    want = dg.linear(Ad, Bd, bias=bd, act="silu", residual=Rd)
    torch.cuda.synchronize()
    bad = []

    def work(s):
        for _ in range(20):
            C = dg.linear(Ad, Bd, bias=bd, act="silu", residual=Rd, stream=s)
            s.synchronize()
            if not torch.equal(C, want):
                bad.append(1)
    threads = [threading.Thread(target=work, args=(torch.cuda.Stream(),)) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_refusals_leave_the_outputs():
    bf = torch.bfloat16
    A, B = torch.zeros(4, 8, dtype=bf, device="cuda"), torch.zeros(8, 16, dtype=bf, device="cuda")
    C = torch.full((4, 16), 3.0, dtype=bf, device="cuda")
    with pytest.raises(TypeError):
        dg.gemm_act(A, B, C, residual=C.float())
    with pytest.raises(ValueError):
        dg.gemm_act(A, B, C, act="tanh")
    with pytest.raises(ValueError):
        dg.gemm_act(A, B, C, bias=torch.zeros(15, device="cuda"))
    with pytest.raises(ValueError):
        dg.gemm_act_bwd(A, B, C, dA=A.clone(), act="silu")
    with pytest.raises(dg.DgemmError):
        dg.gemm_act_bwd(A, B, C, dA=A.clone(), act="silu", preact=C.clone())   # no workspace
    with pytest.raises(TypeError):
        dg.gemm_f8(A, A, C[:, :4], torch.ones(4, device="cuda"), torch.ones(4, device="cuda"))
    torch.cuda.synchronize()
    assert bool((C == 3).all())


def test_long_pitch_offsets_past_32_bits():
    """Rows far apart: offsets of whole operands pass 2^32 bytes while each panel
    of 256 rows stays below 2^31."""
    M, N, K, pitch = 1100, 24, 40, 4000 * 1000
    A, B, b, R = inputs(M, N, K, torch.bfloat16, 14)
    big = torch.empty(M * pitch, dtype=torch.bfloat16, device="cuda")  # 8.8 GB
    Ad = torch.as_strided(big, (M, K), (pitch, 1))
    Rd = torch.as_strided(big, (M, N), (pitch, 1), 64)
    Cd = torch.as_strided(big, (M, N), (pitch, 1), 128)
    Ad.copy_(A)
    Rd.copy_(R)
    want = dg.linear(padded(A, torch.bfloat16), padded(B, torch.bfloat16), bias=b.cuda(), act="silu",
                     residual=padded(R, torch.bfloat16))
    dg.gemm_act(Ad, padded(B, torch.bfloat16), Cd, bias=b.cuda(), act="silu", residual=Rd)
    assert torch.equal(Cd, want)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=str)
def test_long_pitch_backward_and_norm(dt):
    """The same for the gradients (products apart and together) and the norm: equal,
    bit for bit, to the calls on compact rows."""
    M, N, K, pitch = 1100, 24, 40, 4000 * 1000 * 2 // dt.itemsize
    A, B, _, dC = inputs(M, N, K, dt, 15)
    Z = torch.randn(M, N, generator=gen(16)).to(dt)
    big = torch.empty(M * pitch, dtype=dt, device="cuda")  # 8.8 GB
    view = lambda cols, at: torch.as_strided(big, (M, cols), (pitch, 1), at)  # noqa: E731
    Ad, dCd, Zd, dAd, Sd = view(K, 0), view(N, 64), view(N, 128), view(K, 192), view(K, 256)
    for d, s in ((Ad, A), (dCd, dC), (Zd, Z)):
        d.copy_(s)
    Ac, dCc, Zc, Bd = (padded(t, dt) for t in (A, dC, Z, B))
    fmt = "f32" if dt == torch.float32 else "bf16"
    work = torch.empty(dg.gemm_act_bwd_workspace(fmt, M, N, K, "silu", dt != torch.float32)[1], dtype=torch.uint8,
                       device="cuda")
    for act in ("silu", "none"):
        for want in ((True, True), (True, False), (False, True)):
            got, ref = [], []
            for a, c, z, da, out in ((Ad, dCd, Zd, dAd, got), (Ac, dCc, Zc, sentinel(M, K, dt), ref)):
                dB = sentinel(K, N, dt) if want[1] else None
                db = torch.full((N,), float("nan"), device="cuda")
                dg.gemm_act_bwd(a, Bd, c, dA=da if want[0] else None, dB=dB, dbias=db, preact=z, act=act,
                                workspace=work)
                out += [t.clone() for t in (da if want[0] else None, dB, db) if t is not None]
            assert all(torch.equal(g, r) for g, r in zip(got, ref)), (act, want)
    w = torch.linspace(0.5, 1.5, K, device="cuda")
    rstd = torch.empty(M, device="cuda")
    dg.rmsnorm(Ad, w, dAd, residual=Ad, total=Sd, rstd=rstd)
    ref = dg.rms_norm(Ac, w, residual=Ac, keep=True)
    assert torch.equal(dAd, ref["Y"]) and torch.equal(Sd, ref["total"]) and torch.equal(rstd, ref["rstd"])
    wsn = torch.empty(dg.rmsnorm_bwd_workspace(M, K), dtype=torch.uint8, device="cuda")
    dw = torch.empty(K, device="cuda")
    dg.rmsnorm_bwd(Ad, Sd, w, rstd, dAd, dtotal=Ad, dweight=dw, workspace=wsn)
    dX, dwr = dg.rms_norm_backward(Ac, ref["total"], w, ref["rstd"], dtotal=Ac)
    assert torch.equal(dAd, dX) and torch.equal(dw, dwr)
