"""The feed-forward block's operators write their outputs and nothing else, and every
workspace ends where the query says."""
import pytest
import torch

import dense_gemm_matrix_amd as dg
from tests.feedforward_ref import blocks
from tests.linear_ref import F8
from tests.test_linear_guards import FILL, Guarded, M_N, WIDTHS, check, grid_plan, rnd, vec, ws  # noqa: F401

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TILES = [None, (16, 32, 1), (16, 64, 2), (32, 32, 1), (64, 64, 1), (128, 128, 1), (128, 128, 2), (256, 256, 1),
         (256, 256, 3)]


def past(buf, n):
    assert bool((buf[n:] == FILL).all())


@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("fmt", list(DT))
@pytest.mark.parametrize("tile", TILES, ids=str)
def test_gated_forward(grid_plan, tile, fmt, out):  # noqa: F811
    dt = DT[fmt]
    od = dt if out == "same" else torch.float32
    if tile:
        grid_plan(*tile)
    for i, (M, N) in enumerate(M_N):
        K = 150
        C, G, U = (Guarded(M, N, od, k) for k in (1, 2, 3))
        n = dg.gemm_gated_plan(fmt, M, N, K, 1 << 30, od == dt)["workspace_bytes"]
        w, buf = ws(n)
        keep = dict(gate=G.t, up=U.t) if i % 2 else {}
        dg.gemm_gated(rnd(M, K, dt), rnd(K, N, dt), rnd(K, N, dt, 1), C.t, bias_g=vec(N), bias_u=vec(N, 1), act="silu",
                      workspace=w, **keep)
        check(C, *((G, U) if keep else ()))
        past(buf, n)


@pytest.mark.parametrize("fmt", list(DT))
@pytest.mark.parametrize("tile", [None, (32, 32, 1), (64, 64, 1), (128, 128, 1), (128, 128, 3), (256, 256, 1),
                                  (256, 256, 2)], ids=str)
def test_gated_backward(grid_plan, tile, fmt):  # noqa: F811
    dt = DT[fmt]
    if tile:
        grid_plan(*tile)
    for M, N in M_N + [(300, 9)]:
        for K in (1, 35, 70):
            for want in ("dA dBg dBu dbias_g dbias_u", "dA", "dBg", "dBu dbias_g", "dbias_u"):
                outs = {"dA": Guarded(M, K, dt), "dBg": Guarded(K, N, dt), "dBu": Guarded(K, N, dt, 2),
                        "dbias_g": Guarded(None, N, torch.float32), "dbias_u": Guarded(None, N, torch.float32)}
                outs = {k: v for k, v in outs.items() if k in want.split()}
                n = dg.gemm_gated_bwd_workspace(fmt, M, N, K)[M % 2]
                w, buf = ws(n)
                dg.gemm_gated_bwd(rnd(M, K, dt), rnd(K, N, dt), rnd(K, N, dt, 1), rnd(M, N, dt, 3), rnd(M, N, dt, 4),
                                  rnd(M, N, dt, 5), act="silu", workspace=w, **{k: v.t for k, v in outs.items()})
                check(*outs.values())
                past(buf, n)


@pytest.mark.parametrize("od", list(DT.values()), ids=str)
@pytest.mark.parametrize("rows_b", [1, 128])
@pytest.mark.parametrize("tile", TILES, ids=str)
def test_f8_block(grid_plan, tile, rows_b, od):  # noqa: F811
    if tile:
        grid_plan(*tile)
    name = [k for k, v in DT.items() if v == od][0]
    for M, N in M_N:
        K = 300
        C = Guarded(M, N, od)
        n = dg.gemm_f8_block_plan(name, M, N, K, 1 << 30, rows_b)["workspace_bytes"]
        w, buf = ws(n)
        sa = torch.rand(M, blocks(K)).cuda() + 0.5
        sb = torch.rand(N if rows_b == 1 else blocks(N), blocks(K)).cuda() + 0.5
        dg.gemm_f8_block(rnd(M, K, F8), rnd(N, K, F8), C.t, sa, sb, bias=vec(N), act="gelu", residual=rnd(M, N, od),
                         workspace=w)
        check(C)
        past(buf, n)


@pytest.mark.parametrize("dt", list(DT.values()), ids=str)
@pytest.mark.parametrize("N", WIDTHS + [20000, 32768])
def test_layer_norm_and_quantizer(N, dt):
    for M in (1, 3, 17):
        X, R, w = rnd(M, N, dt), rnd(M, N, dt, 1), vec(N)
        for f8 in (None, "row", "block"):
            Y, S = Guarded(M, N, F8 if f8 else dt), Guarded(M, N, dt, 2)
            mean, rstd = Guarded(None, M, torch.float32), Guarded(None, M, torch.float32)
            scale = Guarded(M, blocks(N), torch.float32) if f8 == "block" else Guarded(None, M, torch.float32)
            dg.layernorm(X, w, vec(N, 1), Y.t, residual=R, total=S.t, scale=scale.t if f8 else None, mean=mean.t,
                         rstd=rstd.t)
            check(Y, S, mean, rstd, *([scale] if f8 else []))
        Y, scale = Guarded(M, N, F8), Guarded(None, blocks(N) * M, torch.float32)
        dg.rmsnorm(X, w, Y.t, scale=scale.t.view(blocks(N), M).t())
        check(Y, scale)
        for rows in (1, 128):
            Q, scale = Guarded(M, N, F8), Guarded(M if rows == 1 else blocks(M), blocks(N), torch.float32)
            dg.quant_f8_block(X, Q.t, scale.t)
            check(Q, scale)
            Q, scale = Guarded(N, M, F8), Guarded(N if rows == 1 else blocks(N), blocks(M), torch.float32)
            dg.quant_f8_block(X, Q.t, scale.t, transpose=True)
            check(Q, scale)


@pytest.mark.parametrize("dt", list(DT.values()), ids=str)
@pytest.mark.parametrize("N", WIDTHS)
def test_layer_norm_backward(N, dt):
    for M in (1, 3, 17, 515):
        if M * N > 1 << 21:
            continue
        dX, dw, db = Guarded(M, N, dt), Guarded(None, N, torch.float32), Guarded(None, N, torch.float32)
        n = dg.layernorm_bwd_workspace(M, N)
        w, buf = ws(n)
        dg.layernorm_bwd(rnd(M, N, dt), rnd(M, N, dt, 1), vec(N), vec(M), vec(M, 1), dX.t, dtotal=rnd(M, N, dt, 2),
                         dweight=dw.t, dbias=db.t, workspace=w)
        check(dX, dw, db)
        past(buf, n)
