"""The linear layer's operators write their outputs and nothing else: every output lies
in a buffer whose bytes around it (the gap of every row, the last one's too, and rows
before and after) have to stay, and every workspace ends where the query says."""
import pytest
import torch

import dense_gemm_matrix_amd as dg
from tests.linear_ref import F8, padded

FILL = 0xA5
GUARD = 8  # rows (or vector elements times 16) on either side


class Guarded:
    """A rows x cols matrix (or a vector of `cols`) inside a buffer of FILL bytes."""

    def __init__(self, rows, cols, dtype, extra=1, device="cuda"):
        es = torch.empty((), dtype=dtype).element_size()
        self.rows, self.row_bytes = max(rows or 1, 0), cols * es
        self.pitch = (self.row_bytes + 15) // 16 * 16 + 16 * extra
        self.buf = torch.full(((self.rows + 2 * GUARD) * self.pitch,), FILL, dtype=torch.uint8, device=device)
        flat = self.buf.view(dtype)
        at = GUARD * self.pitch // es
        self.t = torch.as_strided(flat, (cols,), (1,), at) if rows is None else \
            torch.as_strided(flat, (rows, cols), (self.pitch // es, 1), at)

    def kept(self):
        b = self.buf.cpu().view(-1, self.pitch)
        inside = torch.zeros_like(b, dtype=torch.bool)
        inside[GUARD:GUARD + self.rows, :self.row_bytes] = True
        return bool((b[~inside] == FILL).all())

    def written(self):
        return not bool((self.buf.view(-1, self.pitch)[GUARD:GUARD + self.rows, :self.row_bytes] == FILL).all())


@pytest.mark.parametrize("rows", [1, 2, 5])
@pytest.mark.parametrize("cols", [1, 3, 8])
def test_guards_see_every_stray_byte(rows, cols):
    g = Guarded(rows, cols, torch.bfloat16, device="cpu")
    assert g.kept() and not g.written()
    g.t.fill_(1.0)
    assert g.kept() and g.written()
    strays = [g.buf.numel() - 1, 0, GUARD * g.pitch - 1, (GUARD + rows) * g.pitch]
    strays += [(GUARD + r) * g.pitch + c for r in range(rows) for c in range(g.row_bytes, g.pitch)]
    for at in strays:
        old = int(g.buf[at])
        g.buf[at] = 7
        assert not g.kept(), at
        g.buf[at] = old
    assert g.kept()


def ws(n):
    """A workspace of exactly n bytes inside a guarded buffer."""
    buf = torch.full((n + 4096,), FILL, dtype=torch.uint8, device="cuda")
    return buf[:n], buf


def rnd(rows, cols, dt, seed=0):
    return padded(torch.randn(rows, cols, generator=torch.Generator().manual_seed(seed + rows + cols)), dt, 1)


def vec(n, seed=0):
    return torch.rand(n, generator=torch.Generator().manual_seed(seed + n)).cuda() + 0.5


def check(*guards):
    torch.cuda.synchronize()
    for g in guards:
        assert g.written() and g.kept()


@pytest.fixture
def grid_plan():
    yield lambda r, c, s: dg.dgemm_set_plan_override(dg.DGEMM_PLAN_GRID, r, c, s)
    dg.dgemm_set_plan_override(dg.DGEMM_PLAN_AUTO)


DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "f32x3": torch.float32}
# few rows, slice-K, grid; one column, odd, a multiple of 8 and past a tile
M_N = [(1, 1), (1, 3), (1, 37), (1, 130), (2, 8), (15, 65), (16, 33), (17, 1), (31, 7), (33, 40), (65, 63), (129, 131)]
TILES = [None, (16, 32, 1), (16, 64, 2), (32, 32, 4), (32, 32, 8), (64, 64, 4), (128, 128, 1), (128, 128, 2),
         (256, 256, 1), (192, 256, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("fmt", list(DT))
@pytest.mark.parametrize("tile", TILES, ids=str)
def test_forward(grid_plan, tile, fmt, out):
    dt = DT[fmt]
    od = dt if out == "same" else torch.float32
    if tile:
        grid_plan(*tile)
    for M, N in M_N:
        K = 150
        C, Z = Guarded(M, N, od), Guarded(M, N, od, 2)
        n = dg.gemm_act_plan(fmt, M, N, K, 1 << 30, od == dt and od != torch.float32)["workspace_bytes"]
        w, buf = ws(n)
        dg.gemm_act(rnd(M, K, dt), rnd(K, N, dt), C.t, bias=vec(N), act="silu", residual=rnd(M, N, od),
                    preact=Z.t, workspace=w, in_fmt=fmt)
        check(C, Z)
        assert bool((buf[n:] == FILL).all())


@pytest.mark.gpu
@pytest.mark.parametrize("od", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("tile", [t for t in TILES if not t or t[0] not in (16, 192)], ids=str)
def test_8_bit_forward(grid_plan, tile, od):
    if tile:
        grid_plan(*tile)
    name = {torch.bfloat16: "bf16", torch.float16: "f16", torch.float32: "f32"}[od]
    for M, N in M_N:
        K = 300
        C = Guarded(M, N, od)
        n = dg.gemm_f8_plan(name, M, N, K, 1 << 30)["workspace_bytes"]
        w, buf = ws(n)
        dg.gemm_f8(rnd(M, K, F8), rnd(N, K, F8), C.t, vec(M), vec(N), bias=vec(N), act="gelu",
                   residual=rnd(M, N, od), workspace=w)
        check(C)
        assert bool((buf[n:] == FILL).all())


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", list(DT))
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("tile", [None, (32, 32, 4), (64, 64, 4), (32, 32, 8), (128, 128, 1), (128, 128, 2),
                                  (256, 256, 1)], ids=str)
def test_backward(grid_plan, tile, act, fmt):
    dt = DT[fmt]
    if tile:
        grid_plan(*tile)
    for M, N in M_N + [(300, 9)]:
        for K in (1, 35, 70):
            for want in ("dA dB dbias", "dA", "dB", "dbias"):
                dA, dB, db = Guarded(M, K, dt), Guarded(K, N, dt), Guarded(None, N, torch.float32)
                outs = {"dA": dA, "dB": dB, "dbias": db}
                outs = {k: v for k, v in outs.items() if k in want.split()}
                req, best = dg.gemm_act_bwd_workspace(fmt, M, N, K, act, fmt[:3] != "f32")
                n = best if M % 2 else req
                w, buf = ws(n)
                dg.gemm_act_bwd(rnd(M, K, dt), rnd(K, N, dt), rnd(M, N, dt, 3),
                                preact=None if act == "none" else rnd(M, N, dt, 4), act=act, workspace=w, in_fmt=fmt,
                                **{k: v.t for k, v in outs.items()})
                check(*outs.values())
                assert bool((buf[n:] == FILL).all())


WIDTHS = [1, 3, 7, 8, 64, 65, 128, 130, 255, 256, 513, 1000, 1024, 1030, 2048, 3001, 4096, 4100, 8190, 9001, 16384]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("N", WIDTHS + [20000, 32768])
def test_norm_and_quantizer(N, dt):
    for M in (1, 3, 17):
        X, R, w = rnd(M, N, dt), rnd(M, N, dt, 1), vec(N)
        for f8 in (False, True):
            Y, S = Guarded(M, N, F8 if f8 else dt), Guarded(M, N, dt, 2)
            rstd, scale = Guarded(None, M, torch.float32), Guarded(None, M, torch.float32)
            dg.rmsnorm(X, w, Y.t, residual=R, total=S.t, scale=scale.t if f8 else None, rstd=rstd.t)
            check(Y, S, rstd, *([scale] if f8 else []))
        Q, scale = Guarded(M, N, F8), Guarded(None, M, torch.float32)
        dg.quant_f8(X, Q.t, scale.t)
        check(Q, scale)
        if N <= 4100:
            Q, scale = Guarded(N, M, F8), Guarded(None, N, torch.float32)
            dg.quant_f8(X, Q.t, scale.t, transpose=True)
            check(Q, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("N", WIDTHS)
def test_norm_backward(N, dt):
    for M in (1, 3, 17, 515):
        if M * N > 1 << 21:
            continue
        dX, dw = Guarded(M, N, dt), Guarded(None, N, torch.float32)
        n = dg.rmsnorm_bwd_workspace(M, N)
        w, buf = ws(n)
        dg.rmsnorm_bwd(rnd(M, N, dt), rnd(M, N, dt, 1), vec(N), vec(M), dX.t, dtotal=rnd(M, N, dt, 2), dweight=dw.t,
                       workspace=w)
        check(dX, dw)
        assert bool((buf[n:] == FILL).all())
