"""gemm_gated and gemm_gated_bwd on the GPU against plain 64-bit forms."""
import threading

import pytest
import torch

import dense_gemm_matrix_amd as dg
from tests.feedforward_ref import H, e4m3, rounded
from tests.linear_ref import SLOPE, act64, act_grad64, gap_kept, padded, sentinel, sum_bound, within

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
FORMS = [("bf16", "same"), ("bf16", "f32"), ("f16", "same"), ("f16", "f32"), ("f32", "f32")]
ACTS = list(dg.ACT_CODES)


@pytest.fixture
def plan():
    """Forces a tile and split count for the test."""
    def force(rows, cols, splits=1):
        dg.dgemm_set_plan_override(dg.DGEMM_PLAN_GRID, rows, cols, splits)
    yield force
    dg.dgemm_set_plan_override(dg.DGEMM_PLAN_AUTO)


def inputs(M, N, K, dt, seed):
    g = torch.Generator().manual_seed(seed)
    A = torch.randn(M, K, generator=g).to(dt)
    Bg, Bu = ((torch.randn(K, N, generator=g) / max(1, K) ** 0.5).to(dt) for _ in range(2))
    return A, Bg, Bu, torch.randn(N, generator=g), torch.randn(N, generator=g)


def space(n):
    return torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda") if n else None


def run(fmt, out, M, N, K, act, seed=0, bias=True, keep=True, ws_bytes=0):
    dt = DT[fmt]
    od = torch.float32 if out == "f32" else dt
    A, Bg, Bu, bg, bu = inputs(M, N, K, dt, seed)
    C = sentinel(M, N, od)
    G, Up = (sentinel(M, N, od, 2), sentinel(M, N, od, 3)) if keep else (None, None)
    dg.gemm_gated(padded(A, dt, 1), padded(Bg, dt, 1), padded(Bu, dt, 3), C, bias_g=bg.cuda() if bias else None,
                  bias_u=bu.cuda() if bias else None, act=act, gate=G, up=Up, workspace=space(ws_bytes))
    torch.cuda.synchronize()
    a = A.double()
    z, d = [], []
    for B, b in ((Bg, bg), (Bu, bu)):
        v, s = a @ B.double(), a.abs() @ B.double().abs()
        if bias:
            v, s = v + b.double(), s + b.double().abs()
        z.append(v)
        d.append(sum_bound(K, s))
    if keep:
        for got, v, e in ((G, z[0], d[0]), (Up, z[1], d[1])):
            within(got, v, rounded(e, v, od))
            assert gap_kept(got)
    # act's slope carries G's error, its own evaluation 32 half steps of |G|; the product one more
    v = act64(z[0], act)
    ea = d[0] if act == "none" else SLOPE * d[0] + 32 * H * z[0].abs()
    want = v * z[1]
    e = z[1].abs() * ea + v.abs() * d[1] + ea * d[1] + H * want.abs() * 2
    within(C, want, rounded(e, want, od))
    assert gap_kept(C)


SHAPES = [(1, 1, 1), (1, 33, 40), (1, 200, 515), (2, 40, 5000), (5, 130, 33), (16, 97, 257), (17, 70, 65), (33, 8, 130),
          (70, 129, 200), (130, 300, 72), (300, 140, 264)]


@pytest.mark.parametrize("fmt, out", FORMS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_forward(fmt, out, shape):
    i = SHAPES.index(shape)
    run(fmt, out, *shape, ACTS[i % 5], seed=i)
    run(fmt, out, *shape, ACTS[(i + 2) % 5], seed=i + 50, bias=False, keep=False)
    run(fmt, out, *shape, ACTS[(i + 4) % 5], seed=i + 70, bias=i % 2 == 0, ws_bytes=16 << 20)


@pytest.mark.parametrize("fmt, tile", [("bf16", 256), ("bf16", 128), ("f16", 256), ("f16", 128), ("f32", 128)])
@pytest.mark.parametrize("splits", [1, 3])
def test_forward_grid_tiles(plan, fmt, tile, splits):
    plan(tile, tile, splits)
    ws = 0 if splits == 1 else 16 << 20
    run(fmt, "same", 300, 270, 200, "gelu_tanh", seed=11, ws_bytes=ws)
    run(fmt, "same", 261, 515, 328, "silu", seed=12, bias=False, ws_bytes=ws)
    run(fmt, "f32", 130, 31, 64, "gelu", seed=13, keep=False, ws_bytes=ws)
    run(fmt, "same", 40, 1030, 1000, "relu", seed=14, ws_bytes=ws)


@pytest.mark.parametrize("fmt", list(DT))
@pytest.mark.parametrize("tile", [32, 64])
def test_forward_slice_tiles(plan, fmt, tile):
    plan(tile, tile)
    for i, (M, N, K) in enumerate([(40, 70, 600), (65, 33, 1290), (17, 200, 130), (100, 129, 64), (33, 31, 30)]):
        run(fmt, "same", M, N, K, ACTS[i % 5], seed=i)
        run(fmt, "f32", M, N, K, ACTS[(i + 2) % 5], seed=i, bias=False, keep=False)


@pytest.mark.parametrize("cols", [32, 64])
@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("fmt", list(DT))
def test_forward_few_row_strips(plan, cols, splits, fmt):
    plan(16, cols, splits)
    ws = 0 if splits == 1 else 4 << 20
    for i, (M, N, K) in enumerate([(1, 300, 1030), (16, 129, 64), (7, 20, 333)]):
        run(fmt, "same", M, N, K, "silu", seed=20 + i, ws_bytes=ws)
        run(fmt, "f32", M, N, K, "none", seed=30 + i, ws_bytes=ws, keep=False)


@pytest.mark.parametrize("fmt", list(DT))
@pytest.mark.parametrize("shape", [(1, 2050, 4130), (16, 500, 4096), (40, 300, 8200)],
                         ids=lambda s: "x".join(map(str, s)))
def test_forward_deep(fmt, shape):
    """The planner's own splits."""
    assert dg.gemm_gated_plan(fmt, *shape, 1 << 30, True)["splits"] > 1
    run(fmt, "same", *shape, "silu", seed=20, ws_bytes=64 << 20)


def test_integers_are_exact():
    for M, N, K in [(1, 70, 100), (16, 40, 64), (40, 72, 96), (300, 264, 200)]:
        g = torch.Generator().manual_seed(M)
        A, Bg, Bu = (torch.randint(-3, 4, s, generator=g).float() for s in ((M, K), (K, N), (K, N)))
        for dt in DT.values():
            C, G, Up = dg.linear_gated(padded(A, dt), padded(Bg, dt), padded(Bu, dt), act="relu", keep_preact=True,
                                       out_dtype=torch.float32)
            assert torch.equal(G.cpu(), A @ Bg) and torch.equal(Up.cpu(), A @ Bu)
            assert torch.equal(C.cpu(), (A @ Bg).clamp_min(0) * (A @ Bu))


def test_halves_of_one_weight_and_of_one_buffer():
    """Both weights as column windows of one matrix, G and U as windows of one buffer: the results of separate ones."""
    M, N, K, dt = 200, 136, 200, torch.bfloat16
    A, Bg, Bu, _, _ = inputs(M, N, K, dt, 3)
    W = torch.cat([Bg, Bu], 1).cuda()
    Ad = padded(A, dt)
    C, G, Up = dg.linear_gated(Ad, padded(Bg, dt), padded(Bu, dt), keep_preact=True)
    buf = torch.empty(M, 2 * N, dtype=dt, device="cuda")
    C2 = torch.empty(M, N, dtype=dt, device="cuda")
    dg.gemm_gated(Ad, W[:, :N], W[:, N:], C2, gate=buf[:, :N], up=buf[:, N:], workspace=space(64 << 20))
    assert torch.equal(C, C2) and torch.equal(buf[:, :N], G) and torch.equal(buf[:, N:], Up)
    dC = torch.randn(M, N, generator=torch.Generator().manual_seed(1)).to(dt).cuda()
    want = dg.linear_gated_backward(Ad, padded(Bg, dt), padded(Bu, dt), dC, G, Up)
    dW, dA = torch.empty_like(W), torch.empty_like(Ad)
    dg.gemm_gated_bwd(Ad, W[:, :N], W[:, N:], dC, buf[:, :N], buf[:, N:], dA=dA, dBg=dW[:, :N], dBu=dW[:, N:],
                      workspace=space(dg.gemm_gated_bwd_workspace("bf16", M, N, K)[1]))
    assert torch.equal(dA, want[0]) and torch.equal(dW[:, :N], want[1]) and torch.equal(dW[:, N:], want[2])


@pytest.mark.parametrize("M", [3, 40, 300])
def test_nonfinite(M):
    """Infinities and NaN of one row, and of one weight's column, reach that row and column alone; those in the row
    padding, past K and past N reach nothing."""
    N, K, dt = 70, 90, torch.bfloat16
    A, Bg, Bu, _, _ = inputs(M, N, K, dt, 1)
    ref = dg.linear_gated(padded(A, dt), padded(Bg, dt), padded(Bu, dt)).float().cpu()
    assert ref.isfinite().all()  # the gaps hold NaN
    A2 = A.clone()
    A2[1, 5] = float("nan")
    Bg2 = Bg.clone()
    Bg2[7, 11] = float("inf")
    C = dg.linear_gated(padded(A2, dt), padded(Bg2, dt), padded(Bu, dt)).float().cpu()
    rows, cols = torch.arange(M) != 1, torch.arange(N) != 11
    assert C[1].isnan().all()
    assert torch.equal(C[rows][:, cols], ref[rows][:, cols]) and not C[rows][:, 11].isfinite().any()


def test_special_gates():
    """silu of +inf is +inf and of -inf NaN, relu passes NaN, as gemm_act's."""
    g = torch.tensor([float("inf"), float("-inf"), float("nan"), -0.0, 3.0])
    eye, one = padded(torch.ones(20, 1), torch.float32), padded(torch.zeros(1, 5), torch.float32)
    for act, want in (("silu", [float("inf"), float("nan"), float("nan"), -0.0]),
                      ("relu", [float("inf"), 0.0, float("nan"), 0.0])):
        for rows in (1, 20):
            C = dg.linear_gated(eye[:rows], one, one, bias_g=g.cuda(), bias_u=torch.full((5,), 2.0).cuda(), act=act)
            assert torch.equal(C[0, :4].cpu().nan_to_num(7.0), torch.tensor(want).nan_to_num(7.0))


# ------------------------------------------------------------------ backward

def run_bwd(fmt, out, M, N, K, act, seed, least=False, want=("dA", "dBg", "dBu", "dbias_g", "dbias_u")):
    dt = DT[fmt]
    cd = torch.float32 if out == "f32" else dt
    A, Bg, Bu, _, _ = inputs(M, N, K, dt, seed)
    g = torch.Generator().manual_seed(seed + 1)
    dC, G, Up = (torch.randn(M, N, generator=g).to(cd) for _ in range(3))
    outs = {"dA": (M, K), "dBg": (K, N), "dBu": (K, N)}
    outs = {k: sentinel(*s, dt) for k, s in outs.items() if k in want}
    outs.update({k: torch.full((N,), float("nan"), device="cuda") for k in ("dbias_g", "dbias_u") if k in want})
    req, best = dg.gemm_gated_bwd_workspace(fmt, M, N, K, cd == dt)
    dg.gemm_gated_bwd(padded(A, dt, 1), padded(Bg, dt, 1), padded(Bu, dt, 2), padded(dC, cd, 1), padded(G, cd, 2),
                      padded(Up, cd, 3), act=act, workspace=space(req if least else best), **outs)
    torch.cuda.synchronize()
    A, Bg, Bu, c, z, u = (t.double() for t in (A, Bg, Bu, dC, G, Up))
    s, v = act_grad64(z, act), act64(z, act)
    # fp32 values: the slope within 32 half steps of 1.13 (of |G| for the activation), two products' roundings
    zg, zu = c * u * s, c * v
    eg = H * (32 * SLOPE * (c * u).abs() + 3 * zg.abs())
    eu = H * (32 * (c * z).abs() + 2 * zu.abs())
    rg, ru = rounded(eg, zg, dt), rounded(eu, zu, dt)  # as the products take them
    if "dA" in want:
        ref = zg @ Bg.t() + zu @ Bu.t()
        b = rg @ Bg.abs().t() + ru @ Bu.abs().t()
        b = b + sum_bound(2 * N, (zg.abs() + rg) @ Bg.abs().t() + (zu.abs() + ru) @ Bu.abs().t())
        within(outs["dA"], ref, rounded(b, ref, dt))
    for k, d, r in (("dBg", zg, rg), ("dBu", zu, ru)):
        if k in want:
            ref = A.t() @ d
            b = A.abs().t() @ r + sum_bound(M, A.abs().t() @ (d.abs() + r))
            within(outs[k], ref, rounded(b, ref, dt))
    for k, d, e in (("dbias_g", zg, eg), ("dbias_u", zu, eu)):
        if k in want:
            within(outs[k], d.sum(0), e.sum(0) + (M + 2) * H * (d.abs() + e).sum(0) + 2.0 ** -149)
    for k in ("dA", "dBg", "dBu"):
        if k in want:
            assert gap_kept(outs[k])
    return outs


BWD_SHAPES = [(1, 1, 1), (1, 33, 40), (16, 130, 97), (5, 515, 200), (17, 70, 65), (33, 8, 130), (70, 129, 200),
              (130, 72, 300), (300, 264, 140), (64, 600, 64)]


@pytest.mark.parametrize("fmt, out", FORMS)
@pytest.mark.parametrize("shape", BWD_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_backward(fmt, out, shape):
    i = BWD_SHAPES.index(shape)
    run_bwd(fmt, out, *shape, ACTS[i % 5], seed=i)
    run_bwd(fmt, out, *shape, ACTS[(i + 3) % 5], seed=i + 9, least=True)


@pytest.mark.parametrize("fmt, tile", [("bf16", 256), ("bf16", 128), ("f16", 256), ("f16", 128)] +
                         [(f, t) for f in DT for t in (32, 64)])
def test_backward_tiles(plan, fmt, tile):
    plan(tile, tile)
    for i, (M, N, K) in enumerate([(300, 270, 200), (130, 515, 328), (65, 31, 64), (200, 40, 300)]):
        run_bwd(fmt, "same", M, N, K, ACTS[i], seed=i)


@pytest.mark.parametrize("fmt, tile", [("bf16", 256), ("bf16", 128), ("f16", 256), ("f16", 128)])
@pytest.mark.parametrize("splits", [2, 3, 7])
def test_backward_in_runs(plan, fmt, tile, splits):
    """Runs of dA's steps that end inside the first pair, at its end and inside the second, and of the batch."""
    for i, (M, N, K) in enumerate([(300, 270, 200), (130, 512, 328), (65, 1000, 64), (40, 449, 300)]):
        plan(tile, tile, splits)
        run_bwd(fmt, "same", M, N, K, ACTS[i], seed=i)
        run_bwd(fmt, "f32", M, N, K, ACTS[i], seed=i, want=("dA", "dBu", "dbias_g"))


@pytest.mark.parametrize("fmt", list(DT))
@pytest.mark.parametrize("shape", [(1, 1100, 40), (16, 1030, 72), (7, 2050, 33), (13, 1025, 1200), (3, 700, 1600)],
                         ids=lambda s: "x".join(map(str, s)))
def test_backward_of_few_rows(fmt, shape):
    """By the kernels for few rows, with the least workspace, and in runs, with more."""
    for least in (True, False):
        run_bwd(fmt, "same", *shape, "silu", seed=5, least=least)
        for want in (("dA",), ("dBg", "dBu"), ("dBu", "dbias_g")):
            run_bwd(fmt, "same", *shape, "gelu", seed=6, least=least, want=want)


@pytest.mark.parametrize("fmt", ["bf16", "f16"])
@pytest.mark.parametrize("shape", [(9000, 520, 136), (4096, 577, 323), (543, 5065, 103)],
                         ids=lambda s: "x".join(map(str, s)))
def test_backward_of_long_batches(fmt, shape):
    """The planner's runs of the batch."""
    req, best = dg.gemm_gated_bwd_workspace(fmt, *shape)
    assert best > req
    run_bwd(fmt, "same", *shape, "silu", seed=7)
    run_bwd(fmt, "f32", *shape, "gelu_tanh", seed=8, want=("dBg",))
    run_bwd(fmt, "same", *shape, "none", seed=9, want=("dBu", "dA"))


def test_backward_of_fp32_by_the_grid():
    """Large enough for transposed copies and the fp32 grid kernels."""
    for i, (M, N, K) in enumerate([(1500, 1100, 1300), (3000, 2000, 260)]):
        run_bwd("f32", "same", M, N, K, "silu", seed=i)
        run_bwd("f32", "same", M, N, K, "silu", seed=i, want=("dA", "dbias_u"))
        run_bwd("f32", "same", M, N, K, "silu", seed=i, want=("dBu",))


@pytest.mark.parametrize("fmt", list(DT))
@pytest.mark.parametrize("M", [7, 200, 700])
def test_backward_parts(fmt, M):
    """Any of the gradients alone."""
    for want in (("dA",), ("dBg",), ("dBu",), ("dBg", "dBu"), ("dbias_g",), ("dbias_u",), ("dA", "dbias_u"),
                 ("dBu", "dbias_g")):
        run_bwd(fmt, "same", M, 300, 264, "silu", seed=4, want=want)


def test_backward_is_the_gradient():
    """Against differences of the forward definition in 64 bits."""
    M, N, K, h = 20, 9, 12, 1e-6
    A, Bg, Bu, bg, bu = (t.double() for t in inputs(M, N, K, torch.float32, 1))
    w = torch.randn(M, N, generator=torch.Generator().manual_seed(9)).double()
    for act in ACTS:
        def loss(a, x, y, p, q):
            return (w * act64(a @ x + p, act) * (a @ y + q)).sum()

        f = [t.float().cuda() for t in (A, Bg, Bu)]
        C, G, Up = dg.linear_gated(*(padded(t.cpu(), torch.float32) for t in f), bias_g=bg.float().cuda(),
                                   bias_u=bu.float().cuda(), act=act, keep_preact=True)
        grads = dg.linear_gated_backward(*(padded(t.cpu(), torch.float32) for t in f), padded(w, torch.float32), G, Up,
                                         act=act, bias=True)
        at = [A, Bg, Bu, bg, bu]
        for i, g in enumerate(grads):
            flat = at[i].reshape(-1)
            for j in (0, flat.numel() // 2, flat.numel() - 1):
                e = torch.zeros_like(flat)
                e[j] = h
                e = e.view(at[i].shape)
                up, dn = [x if k != i else x + e for k, x in enumerate(at)], [x if k != i else x - e for k, x in enumerate(at)]
                num = float((loss(*up) - loss(*dn)) / (2 * h))
                # fp32's sums of up to 20 terms of a few units each, and h^2
                assert abs(num - float(g.cpu().double().reshape(-1)[j])) < 1e-4, (act, i, j)


def test_empty():
    a, b = torch.empty(0, 8, device="cuda"), torch.randn(8, 12, device="cuda")
    C, G, Up = dg.linear_gated(a, b, b, keep_preact=True)
    assert C.shape == G.shape == Up.shape == (0, 12)
    out = dg.linear_gated_backward(a, b, b, C, G, Up, bias=True)
    assert out[0].shape == (0, 8) and all((t == 0).all() and t.numel() for t in out[1:])
    bias = torch.randn(12, device="cuda")
    for M in (4, 40):
        a, w = torch.empty(M, 8, device="cuda")[:, :0], torch.empty(0, 12, device="cuda")
        C = dg.linear_gated(a, w, w, bias_g=bias, bias_u=bias, act="relu")
        assert torch.equal(C, (bias.clamp_min(0) * bias).expand(M, 12))
        a, w = torch.randn(M, 8, device="cuda"), torch.empty(8, 4, device="cuda")[:, :0]
        z = torch.empty(M, 4, device="cuda")[:, :0]
        assert (dg.linear_gated_backward(a, w, w, z, z, z)[0] == 0).all()


def test_refusals():
    A, B, C = torch.zeros(20, 16, device="cuda"), torch.zeros(16, 24, device="cuda"), torch.zeros(20, 24, device="cuda")
    for args, kw in [((A, B, B[:, :20], C), {}), ((A, B, B.bfloat16(), C), {}), ((A, B, B.cpu(), C), {}),
                     ((A, B, None, C), {}), ((A, B, B, C[:19]), {}), ((A, B, B, C.bfloat16()), {}),
                     ((A, B, B, C), dict(act="swish")), ((A, B, B, C), dict(gate=C[:, :20])),
                     ((A, B, B, C), dict(bias_g=C[0, :20])), ((e4m3(20, 16, seed=1).cuda(), B, B, C), {})]:
        with pytest.raises((ValueError, TypeError)):
            dg.gemm_gated(*args, **kw)
    for kw in (dict(gate=C), dict(up=C)):
        with pytest.raises(dg.DgemmError):
            dg.gemm_gated(A, B, B, C, **kw)
    with pytest.raises(dg.DgemmError):
        dg.gemm_gated_bwd(A, B, B, C, C, C, dA=torch.empty_like(A))  # no workspace
    for args in ((A, B, B, C, None, C), (A, B, B, C, C, C[:, :20]), (A, B, None, C, C, C)):
        with pytest.raises(ValueError):
            dg.gemm_gated_bwd(*args)
    # the same matrix as both weights, and as both factors, is an input like any other
    got = dg.linear_gated(A + 1, B + 1, B + 1, act="none")
    assert (got == 256).all()


def test_streams_threads_and_the_same_bits():
    """Calls from several threads on streams of their own give the bits of a call alone."""
    M, N, K, dt = 300, 264, 520, torch.bfloat16
    A, Bg, Bu, _, _ = (t.cuda() for t in inputs(M, N, K, dt, 3))
    want = dg.linear_gated(A, Bg, Bu, keep_preact=True)
    grads = dg.linear_gated_backward(A, Bg, Bu, want[0], *want[1:], bias=True)
    torch.cuda.synchronize()
    bad = []

    def work():
        s = torch.cuda.Stream()
        for _ in range(5):
            got = dg.linear_gated(A, Bg, Bu, keep_preact=True, stream=s)
            g = dg.linear_gated_backward(A, Bg, Bu, got[0], *got[1:], bias=True, stream=s)
            s.synchronize()
            if not all(torch.equal(x, y) for x, y in zip((*got, *g), (*want, *grads))):
                bad.append(1)

    threads = [threading.Thread(target=work) for _ in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad


@pytest.mark.parametrize("M", [3, 200])
def test_captured(M):
    N, K, dt = 264, 2100, torch.bfloat16
    A, Bg, Bu, bg, bu = (t.cuda() for t in inputs(M, N, K, dt, 3))
    A, Bg, Bu = (padded(t.cpu(), dt) for t in (A, Bg, Bu))

    def step():
        C, G, Up = dg.linear_gated(A, Bg, Bu, bias_g=bg, bias_u=bu, keep_preact=True)
        return [C, G, Up, *dg.linear_gated_backward(A, Bg, Bu, C, G, Up, bias=True)]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(3):
        A.copy_(inputs(M, N, K, dt, 20 + i)[0])
        want = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i
