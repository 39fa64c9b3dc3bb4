"""gemm_f8_block and quant_f8_block on the GPU against plain 64-bit forms."""
import pytest
import torch

import dense_gemm_matrix_amd as dg
from tests.feedforward_ref import block_bound, block_product64, blocks, e4m3, quant_block64, spread
from tests.linear_ref import F8, act64, gap_kept, out_bound, padded, sentinel, within

pytestmark = pytest.mark.gpu

DTS = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture
def grid_plan():
    """Forces a tile and split count for the test."""
    def force(rows, cols, splits=1):
        dg.dgemm_set_plan_override(dg.DGEMM_PLAN_GRID, rows, cols, splits)
    yield force
    dg.dgemm_set_plan_override(dg.DGEMM_PLAN_AUTO)


# ------------------------------------------------------------------ the quantizer

QSIZES = [(1, 1), (1, 128), (3, 127), (130, 129), (5, 1000), (128, 128), (129, 257), (300, 515), (2, 9001), (700, 72)]


def scale_views(rows, cols):
    """Scales with neighbouring rows, neighbouring blocks, and padding between both."""
    yield torch.full((cols, rows), float("nan"), device="cuda").t()
    yield torch.full((rows, cols), float("nan"), device="cuda")
    yield torch.full((rows, 2 * cols + 3), float("nan"), device="cuda")[:, ::2][:, :cols]


@pytest.mark.parametrize("dt", DTS, ids=str)
@pytest.mark.parametrize("size", QSIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("rows, transpose", [(1, False), (128, False), (1, True), (128, True)])
def test_quantizer_is_exact(dt, size, rows, transpose):
    M, N = size
    g = torch.Generator().manual_seed(M + N)
    X = (torch.randn(M, N, generator=g) * torch.exp(2 * torch.randn(M, 1, generator=g))).to(dt)
    if M > 2:
        X[1] = 0
        X[2, : N // 2] *= 1e-3
    want, scale = quant_block64(X.t() if transpose else X, rows)
    for sc in scale_views(*scale.shape):
        Q = sentinel(*want.shape, F8)
        dg.quant_f8_block(padded(X, dt, 1), Q, sc, transpose=transpose)
        torch.cuda.synchronize()
        assert torch.equal(sc.cpu(), scale)
        assert torch.equal(Q.cpu().double(), want)
        assert gap_kept(Q)


def test_quantizer_many_rows():
    """Enough blocks for the variant with four in flight, short last workgroups and blocks."""
    X = torch.randn(2111, 1100, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    Q, sc = dg.quantize_f8_block(padded(X, X.dtype))
    want, scale = quant_block64(X, 1)
    assert torch.equal(sc.cpu(), scale) and torch.equal(Q.cpu().double(), want)


def test_quantizer_rounds_once():
    """Values an fp32 quotient puts on the border between two codes, though they lie beside it: x = border * s moved by
    one step of fp32."""
    s = torch.tensor(1.0) / 448 * 7.3  # the scale of a block whose largest is 7.3
    scale = torch.tensor(7.3) / torch.tensor(448.0)
    borders = torch.tensor([17.0 / 16, 19.0 / 16, 5.0 * 2 ** -10, 433.0 / 1, 27 / 16 * 32.0, 29 / 16 * 8.0])
    near = (borders.double() * scale.double()).float()
    x = torch.cat([torch.tensor([7.3]), near, torch.nextafter(near, near * 2), torch.nextafter(near, near * 0),
                   -near, -torch.nextafter(near, near * 2)])
    X = torch.zeros(128)
    X[: x.numel()] = x
    X = X[None]
    want, sc = quant_block64(X, 1)
    for tr, rows, inp in ((False, 1, X), (True, 1, X.t().contiguous()), (False, 128, X)):
        Q, got = dg.quantize_f8_block(padded(inp, torch.float32), rows=rows, transpose=tr)
        assert torch.equal(got.cpu(), sc), s
        assert torch.equal(Q.cpu().double(), want)


@pytest.mark.parametrize("rows, transpose", [(1, False), (128, False), (1, True), (128, True)])
def test_quantizer_nonfinite_blocks(rows, transpose):
    """A block with an infinity or a NaN has scale NaN, all others are what they are without it."""
    X = torch.randn(200, 300, generator=torch.Generator().manual_seed(2))
    for bad in (float("inf"), float("nan")):
        Z = X.clone()
        Z[130, 140] = bad
        q0, s0 = dg.quantize_f8_block(padded(X, X.dtype), rows=rows, transpose=transpose)
        q1, s1 = dg.quantize_f8_block(padded(Z, Z.dtype), rows=rows, transpose=transpose)
        i, j = (140, 130) if transpose else (130, 140)
        hit = torch.zeros(s0.shape, dtype=torch.bool)
        hit[i // rows, j // 128] = True
        assert s1.cpu()[hit].isnan().all() and torch.equal(s1.cpu()[~hit], s0.cpu()[~hit])
        clean = spread(hit.float(), rows, *q0.shape) == 0
        assert torch.equal(q1.cpu().float()[clean], q0.cpu().float()[clean])


# ------------------------------------------------------------------ the product

def inputs(M, N, K, rows_b, seed):
    g = torch.Generator().manual_seed(seed)
    A, B = e4m3(M, K, seed=seed), e4m3(N, K, seed=seed + 1)
    sa = torch.exp(torch.randn(M, blocks(K), generator=g)) / 60
    sb = torch.exp(torch.randn(-(-N // rows_b), blocks(K), generator=g)) / 60 / max(K, 1) ** 0.5
    return A, B, sa, sb, torch.randn(N, generator=g), torch.randn(M, N, generator=g)


def run(M, N, K, od, rows_b, act="none", seed=0, bias=False, residual=False, ws_bytes=0, by_row=False):
    A, B, sa, sb, b, R = inputs(M, N, K, rows_b, seed)
    R = R.to(od) if residual else None
    C = sentinel(M, N, od)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device="cuda") if ws_bytes else None
    put = (lambda s: s.cuda()) if by_row else (lambda s: s.t().contiguous().cuda().t())
    dg.gemm_f8_block(padded(A, F8, 1), padded(B, F8, 2), C, put(sa), put(sb), bias=b.cuda() if bias else None, act=act,
                     residual=None if R is None else padded(R, od, 1), workspace=ws)
    torch.cuda.synchronize()
    Z, S, drop = block_product64(A, B, sa, sb, rows_b)
    if bias:
        Z, S = Z + b.double(), S + b.double().abs()
    C64 = act64(Z, act)
    C64 = C64 if R is None else C64 + R.double()
    dz = block_bound(K, S)
    if od != torch.float32 and M > 16:
        dz = dz + drop
    within(C, C64, out_bound(C64, Z, dz, R, od, act))
    assert gap_kept(C)


SHAPES = [(1, 1, 1), (1, 130, 300), (16, 33, 129), (5, 16, 1024), (3, 300, 2100), (17, 40, 100), (64, 64, 64),
          (130, 300, 257), (257, 270, 515)]


@pytest.mark.parametrize("od", DTS, ids=str)
@pytest.mark.parametrize("rows_b", [1, 128])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_product(od, rows_b, shape):
    acts = list(dg.ACT_CODES)
    i = SHAPES.index(shape)
    run(*shape, od, rows_b, acts[i % 5], seed=i, bias=True, residual=True)
    run(*shape, od, rows_b, acts[(i + 3) % 5], seed=i, bias=i % 2 == 0, residual=i % 2 == 1, by_row=True)


@pytest.mark.parametrize("tile", [128, 256])
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("rows_b", [1, 128])
def test_grid_tiles(grid_plan, tile, splits, rows_b):
    grid_plan(tile, tile, splits)
    ws = 0 if splits == 1 else 8 << 20
    for i, (M, N, K) in enumerate([(300, 270, 600), (261, 515, 1000), (130, 31, 128), (17, 513, 96)]):
        run(M, N, K, torch.bfloat16, rows_b, "silu", seed=i, bias=True, residual=True, ws_bytes=ws)
        run(M, N, K, torch.float16, rows_b, seed=i, ws_bytes=ws)
        run(M, N, K, torch.float32, rows_b, "gelu", seed=i, residual=True, ws_bytes=ws)


@pytest.mark.parametrize("tile", [32, 64])
@pytest.mark.parametrize("rows_b", [1, 128])
def test_slice_tiles(grid_plan, tile, rows_b):
    grid_plan(tile, tile)
    for i, (M, N, K) in enumerate([(40, 70, 600), (65, 33, 1290), (17, 200, 130), (100, 129, 128)]):
        for od in DTS:
            run(M, N, K, od, rows_b, "silu", seed=i, bias=True, residual=i % 2 == 0)


@pytest.mark.parametrize("shape", [(400, 500, 2048), (1030, 700, 900), (2100, 1100, 400), (250, 260, 65500)], ids=lambda s: "x".join(map(str, s)))
def test_planned_with_a_workspace(shape):
    for od in DTS:
        run(*shape, od, 128, "gelu_tanh", seed=3, bias=True, ws_bytes=64 << 20)


def test_integers_are_exact():
    """Small integers and scales that are powers of two: every sum is exact."""
    for M, N, K in [(1, 70, 300), (16, 40, 64), (40, 72, 200), (300, 264, 520)]:
        g = torch.Generator().manual_seed(M)
        A = torch.randint(-4, 5, (M, K), generator=g).float()
        B = torch.randint(-4, 5, (N, K), generator=g).float()
        sa = torch.exp2(torch.randint(-2, 3, (M, blocks(K)), generator=g).float())
        for rows_b in (1, 128):
            sb = torch.exp2(torch.randint(-2, 3, (-(-N // rows_b), blocks(K)), generator=g).float())
            for od in (torch.float32, torch.bfloat16):
                C = dg.matmul_f8_block(padded(A, F8), padded(B, F8), sa.cuda(), sb.cuda(), out_dtype=od)
                want = (A.double() * spread(sa, 1, M, K)) @ (B.double() * spread(sb, rows_b, N, K)).t()
                assert torch.equal(C.cpu(), want.to(od))


@pytest.mark.parametrize("M", [5, 20, 300])
def test_nan_scales_and_values_keep_to_their_rows(M):
    N, K = 270, 300
    A, B, sa, sb, _, _ = inputs(M, N, K, 128, 1)
    ref = dg.matmul_f8_block(padded(A, F8), padded(B, F8), sa.cuda(), sb.cuda()).float().cpu()
    sa[3, 1] = float("nan")
    C = dg.matmul_f8_block(padded(A, F8), padded(B, F8), sa.cuda(), sb.cuda()).float().cpu()
    rows = torch.arange(M) != 3
    assert C[3].isnan().all() and torch.equal(C[rows], ref[rows])
    sa[3, 1] = 1.0
    sb[1, 2] = float("nan")
    C = dg.matmul_f8_block(padded(A, F8), padded(B, F8), sa.cuda(), sb.cuda()).float().cpu()
    assert C[:, 128:256].isnan().all() and not C[:, :128].isnan().any() and not C[:, 256:].isnan().any()


def test_residual_in_place_and_rows_around():
    for M in (7, 40, 300):
        N, K = 200, 260
        A, B, sa, sb, _, R = inputs(M, N, K, 128, 9)
        R = padded(R, torch.bfloat16, 1)
        want = dg.matmul_f8_block(padded(A, F8), padded(B, F8), sa.cuda(), sb.cuda(), residual=R)
        buf = torch.full((M + 2, 208), 7.0, dtype=torch.bfloat16, device="cuda")
        buf[1:-1, :N] = R
        C = buf[1:-1, :N]
        dg.gemm_f8_block(padded(A, F8), padded(B, F8), C, sa.cuda(), sb.cuda(), residual=C)
        torch.cuda.synchronize()
        assert torch.equal(C, want)
        buf[1:-1, :N] = 7.0
        assert (buf == 7.0).all()


def test_empty():
    e = torch.empty(0, 16, dtype=F8, device="cuda")
    b, s = e4m3(8, 16, seed=1).cuda(), torch.ones(1, 1, device="cuda")
    assert dg.matmul_f8_block(e, b, torch.empty(0, 1, device="cuda"), s).shape == (0, 8)
    none = torch.empty(8, 16, dtype=F8, device="cuda")[:, :0]
    bias = torch.randn(8, device="cuda")
    for M in (8, 40):  # no terms: the bias
        a0 = torch.empty(M, 16, dtype=F8, device="cuda")[:, :0]
        C = dg.matmul_f8_block(a0, none, torch.empty(M, 0, device="cuda"), torch.empty(1, 0, device="cuda"), bias=bias,
                               out_dtype=torch.float32)
        assert torch.equal(C, bias.expand(M, 8))
    Q, sc = dg.quantize_f8_block(torch.empty(0, 16, device="cuda"))
    assert Q.shape == (0, 16) and sc.shape == (0, 1)


def test_a_layer_forward_and_backward():
    """A linear layer in 8 bits with block scales: its product, its input's gradient from the weight's transpose, its
    weight's gradient from both operands quantized along the batch, each against the products of what the codes stand
    for."""
    M, N, K = 384, 260, 520
    g = torch.Generator().manual_seed(5)
    x, W = torch.randn(M, K, generator=g).bfloat16(), (torch.randn(K, N, generator=g) / K ** 0.5).bfloat16()
    dz = (torch.randn(M, N, generator=g) * 0.1).bfloat16()
    xd, Wd, dzd = padded(x, x.dtype), padded(W, W.dtype), padded(dz, dz.dtype)
    xq, xs = dg.quantize_f8_block(xd)
    wq, ws = dg.quantize_f8_block(Wd, rows=128, transpose=True)     # N x K
    wtq, wts = dg.quantize_f8_block(Wd, rows=128)                   # K x N
    assert torch.equal(wts, ws.t()) and torch.equal(wtq.float(), wq.float().t())
    zq, zs = dg.quantize_f8_block(dzd)
    xtq, xts = dg.quantize_f8_block(xd, transpose=True)             # K x M
    ztq, zts = dg.quantize_f8_block(dzd, transpose=True)            # N x M
    for (a, sa, b, sb, rows) in ((xq, xs, wq, ws, 128), (zq, zs, wtq, wts, 128), (xtq, xts, ztq, zts, 1)):
        for od in (torch.bfloat16, torch.float32):
            C = dg.matmul_f8_block(a, b, sa, sb, out_dtype=od)
            Z, S, drop = block_product64(a.cpu(), b.cpu(), sa.cpu(), sb.cpu(), rows)
            dzb = block_bound(a.shape[1], S) + (drop if od != torch.float32 else 0)
            within(C, Z, out_bound(Z, Z, dzb, None, od, "none"))
    # and near the layer's own values: two roundings to e4m3 of at most 2^-4 of a block's value each
    C = dg.matmul_f8_block(xq, wq, xs, ws, out_dtype=torch.float32).cpu().double()
    want = x.double() @ W.double()
    assert float((C - want).norm() / want.norm()) < 2 * 2.0 ** -4


def test_captured_and_on_another_stream():
    M, N, K = 300, 260, 700
    x = padded(torch.randn(M, K, generator=torch.Generator().manual_seed(1)).bfloat16(), torch.bfloat16)
    B, sb = e4m3(N, K, seed=2), torch.rand(blocks(N), blocks(K)) + 0.5
    B, sb = padded(B, F8), sb.cuda()

    def step(stream=None):
        q, s = dg.quantize_f8_block(x, stream=stream)
        return [dg.matmul_f8_block(q, B, s, sb, stream=stream), dg.matmul_f8_block(q[:3], B, s[:3], sb, stream=stream)]

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        x.copy_(torch.randn(M, K, generator=torch.Generator().manual_seed(10 + i)))
        want = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


def test_refusals():
    A, B = e4m3(40, 256, seed=1).cuda(), e4m3(140, 256, seed=2).cuda()
    C = torch.empty(40, 144, device="cuda", dtype=torch.bfloat16)[:, :140]
    sa, sb = torch.ones(40, 2, device="cuda"), torch.ones(2, 2, device="cuda")
    dg.gemm_f8_block(A, B, C, sa, sb)
    for bad in (dict(scale_a=sa[:39]), dict(scale_a=sa[:, :1]), dict(scale_a=sa.double()), dict(scale_a=sa.cpu()),
                dict(scale_b=sb[:1]), dict(scale_b=torch.ones(3, 2, device="cuda")), dict(scale_b=None),
                dict(B=B[:, :240]), dict(A=A.float()), dict(C=C[:39])):
        kw = dict(A=A, B=B, C=C, scale_a=sa, scale_b=sb)
        kw.update(bad)
        with pytest.raises((ValueError, TypeError)):
            dg.gemm_f8_block(*kw.values())
    with pytest.raises(dg.DgemmError):
        dg.gemm_f8_block(A, A[:40], A.view(torch.bfloat16)[:, :40], sa, sa)  # C over A
    X = torch.zeros(40, 256, device="cuda")
    with pytest.raises(dg.DgemmError):
        dg.quant_f8_block(X, A, torch.ones(1, 1, device="cuda").expand(40, 2))
    for bad in (torch.ones(41, 2), torch.ones(40, 3), torch.ones(40)):
        with pytest.raises(ValueError):
            dg.quant_f8_block(X, A, bad.cuda())
    # broadcast scales are inputs like any other
    dg.gemm_f8_block(A, B, C, sa[:1].expand(40, 2), sb[:1, :1].expand(2, 2))
