"""The feed-forward block's entry points on the CPU: refusals come before any device call, plans are reported
without a GPU, and the plain forms the GPU tests use agree with autograd and with torch's own rounding."""
import ctypes
import inspect

import pytest
import torch

import dense_gemm_matrix_amd as dg
from tests.feedforward_ref import layer64, layer_grad64, quant_block64
from tests.linear_ref import F8

V = ctypes.c_void_p
PA, PB, PC, PR, PZ, PW = (0x10000000 * i for i in range(1, 7))
FAR = 0x7000000000
lib = dg.raw()
INVALID, LEADING, MISALIGNED, ALIAS, LARGE, SPACE = (
    dg.DGEMM_ERR_INVALID_VALUE, dg.DGEMM_ERR_LEADING_DIM, dg.DGEMM_ERR_MISALIGNED, dg.DGEMM_ERR_ALIAS,
    dg.DGEMM_ERR_TOO_LARGE, dg.DGEMM_ERR_WORKSPACE)


def without_gpu():
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU: the pointers are made up")


def block_call(out=1, rows=128, M=8, N=8, K=8, A=PA, lda=64, B=PB, ldb=64, C=PC, ldc=64, sa=PR, sar=1, sab=8,
               sb=PR + 256, sbr=1, sbb=1, bias=None, act=0, R=None, ldr=64, ws=None, ws_bytes=0):
    return lib.gemm_f8_block(out, rows, M, N, K, V(A), lda, V(B), ldb, V(C), ldc, V(sa), sar, sab, V(sb), sbr, sbb,
                             V(bias), act, V(R), ldr, V(ws), ws_bytes, None)


@pytest.mark.parametrize("want, kw", [
    (INVALID, dict(out=3)), (INVALID, dict(out=-1)), (INVALID, dict(rows=64)), (INVALID, dict(act=5)),
    (INVALID, dict(N=-1)), (INVALID, dict(sa=0)), (INVALID, dict(sb=0)), (INVALID, dict(B=0)),
    (INVALID, dict(ws_bytes=16)), (LEADING, dict(lda=0)), (LEADING, dict(K=80)), (LEADING, dict(sar=-1)),
    (LEADING, dict(sbb=-4)), (LEADING, dict(R=PZ, ldr=4)), (MISALIGNED, dict(lda=72)), (MISALIGNED, dict(B=PB + 8)),
    (MISALIGNED, dict(sa=PR + 2)), (MISALIGNED, dict(bias=PZ + 2)), (MISALIGNED, dict(R=PZ + 4)),
    (LARGE, dict(lda=1 << 23)), (LARGE, dict(sar=1 << 21)), (LARGE, dict(rows=1, sbr=1 << 21)),
    (ALIAS, dict(C=PA)), (ALIAS, dict(C=PB)), (ALIAS, dict(sa=PC)), (ALIAS, dict(sa=PC - 4 * 7, sar=1)),
    (ALIAS, dict(R=PC + 128)), (ALIAS, dict(R=PC, ldr=72)), (ALIAS, dict(bias=PC)),
    (ALIAS, dict(M=256, N=256, K=65536, lda=65536, ldb=65536, ldc=256, sab=256, sbb=4, B=FAR, C=2 * FAR, ws=FAR,
                 ws_bytes=1 << 40)),
])
def test_gemm_f8_block_refusals(want, kw):
    assert block_call(**kw) == want


def test_gemm_f8_block_accepts_until_the_device():
    without_gpu()
    for kw in (dict(), dict(R=PC), dict(sar=0, sab=0), dict(rows=1), dict(R=PZ, bias=PW), dict(K=0)):
        assert block_call(**kw) == dg.DGEMM_ERR_DEVICE
    assert block_call(M=0, A=0, sa=0, sb=0) == dg.DGEMM_OK and block_call(N=0, B=0, sb=0, sa=0) == dg.DGEMM_OK


def quant_call(in_=1, rows=1, tr=0, M=4, N=200, X=PA, ldx=200, Q=PC, ldq=208, scale=PR, sr=1, sb=4):
    return lib.quant_f8_block(in_, rows, tr, M, N, V(X), ldx, V(Q), ldq, V(scale), sr, sb, None)


@pytest.mark.parametrize("want, kw", [
    (INVALID, dict(in_=3)), (INVALID, dict(rows=2)), (INVALID, dict(tr=2)), (INVALID, dict(M=-1)),
    (INVALID, dict(scale=0)), (INVALID, dict(Q=0)), (LEADING, dict(ldq=192)), (LEADING, dict(ldx=192)),
    (LEADING, dict(sb=3)), (LEADING, dict(sr=0)), (LEADING, dict(sb=0)), (LEADING, dict(sr=-1)),
    (MISALIGNED, dict(Q=PC + 8)), (MISALIGNED, dict(scale=PR + 2)), (MISALIGNED, dict(ldx=201)),
    (LARGE, dict(sr=1 << 21, sb=1 << 25)), (LARGE, dict(rows=128, M=1 << 24, N=12800, ldx=12800, ldq=12800, sr=1, sb=1 << 17)),
    (ALIAS, dict(Q=PA)), (ALIAS, dict(scale=PC)), (ALIAS, dict(scale=PA + 4)),
])
def test_quant_f8_block_refusals(want, kw):
    assert quant_call(**kw) == want


def test_quant_f8_block_accepts_until_the_device():
    without_gpu()
    for kw in (dict(), dict(sr=2, sb=1), dict(sr=5, sb=2), dict(rows=128), dict(tr=1, ldq=16, sr=1, sb=200),
               dict(tr=1, rows=128, ldq=16, sb=2), dict(M=1, sr=0, sb=1)):
        assert quant_call(**kw) == dg.DGEMM_ERR_DEVICE, kw
    assert quant_call(M=0, X=0, Q=0, scale=0) == dg.DGEMM_OK


def norm_call(in_=1, out=0, M=4, N=64, X=PA, ldx=64, R=None, ldr=64, S=None, lds=64, w=PW, b=None, eps=1e-6, Y=PC,
              ldy=64, scale=None, sr=1, sb=4, mean=None, rstd=None):
    return lib.layernorm(in_, out, M, N, V(X), ldx, V(R), ldr, V(S), lds, V(w), V(b), eps, V(Y), ldy, V(scale), sr, sb,
                         V(mean), V(rstd), None)


@pytest.mark.parametrize("want, kw", [
    (INVALID, dict(in_=3)), (INVALID, dict(out=3)), (INVALID, dict(w=0)), (INVALID, dict(eps=-1.0)),
    (INVALID, dict(eps=float("nan"))), (INVALID, dict(out=1)), (INVALID, dict(out=2)), (INVALID, dict(scale=PR)),
    (INVALID, dict(Y=0)), (LEADING, dict(ldx=56)), (LEADING, dict(out=2, scale=PR, sr=0)),
    (LEADING, dict(out=2, scale=PR, N=256, ldx=256, ldy=256, sb=3)), (MISALIGNED, dict(w=PW + 4)),
    (MISALIGNED, dict(b=PZ + 8)), (MISALIGNED, dict(Y=PC + 8)), (MISALIGNED, dict(mean=PR + 2)),
    (LARGE, dict(N=32776, ldx=32776, ldy=32776, Y=FAR)), (ALIAS, dict(Y=PA + 128)), (ALIAS, dict(S=PC)),
    (ALIAS, dict(Y=PW)), (ALIAS, dict(b=PC)), (ALIAS, dict(out=1, scale=PR, Y=PA)), (ALIAS, dict(mean=PA)),
    (ALIAS, dict(mean=PR, rstd=PR)), (ALIAS, dict(out=2, scale=PR, mean=PR + 8)), (ALIAS, dict(R=PR, Y=PR, ldr=128)),
])
def test_layernorm_refusals(want, kw):
    assert norm_call(**kw) == want


def test_layernorm_accepts_until_the_device():
    without_gpu()
    for kw in (dict(), dict(Y=PA), dict(R=PR, S=PR, Y=PA), dict(b=PZ, mean=PB, rstd=PB + 64), dict(out=1, scale=PR),
               dict(out=2, scale=PR), dict(out=1, scale=PR, sr=0, sb=0)):
        assert norm_call(**kw) == dg.DGEMM_ERR_DEVICE, kw
    assert norm_call(M=0, X=0, Y=0) == dg.DGEMM_OK
    assert lib.rmsnorm(1, 2, 4, 64, V(PA), 64, None, 64, None, 64, V(PW), 1e-6, V(PC), 64, V(PR), None, None) \
        == dg.DGEMM_ERR_DEVICE


def bwd_call(in_=1, M=4, N=64, dY=PA, S=PB, w=PW, mean=PR, rstd=PR + 64, dS=None, dX=PC, lddx=64, dw=None, db=None,
             ws=None, ws_bytes=0, ld=64):
    return lib.layernorm_bwd(in_, M, N, V(dY), ld, V(S), ld, V(w), V(mean), V(rstd), V(dS), ld, V(dX), lddx, V(dw),
                             V(db), V(ws), ws_bytes, None)


@pytest.mark.parametrize("want, kw", [
    (INVALID, dict(in_=4)), (INVALID, dict(w=0)), (INVALID, dict(mean=0)), (INVALID, dict(rstd=0)),
    (INVALID, dict(dX=0)), (LEADING, dict(lddx=8)), (MISALIGNED, dict(dY=PA + 2)), (SPACE, dict(dw=PZ)),
    (SPACE, dict(db=PZ, ws=FAR, ws_bytes=255)), (LARGE, dict(N=16392, ld=16392, lddx=16392, S=FAR, dX=2 * FAR)),
    (ALIAS, dict(dX=PB)), (ALIAS, dict(dX=PA + 128)), (ALIAS, dict(dw=PA, ws=FAR, ws_bytes=1 << 20)),
    (ALIAS, dict(dw=PZ, db=PZ, ws=FAR, ws_bytes=1 << 20)), (ALIAS, dict(db=PR, ws=FAR, ws_bytes=1 << 20)),
    (ALIAS, dict(db=PZ, ws=PC, ws_bytes=1 << 20)),
])
def test_layernorm_bwd_refusals(want, kw):
    assert bwd_call(**kw) == want


def test_plans():
    assert dg.gemm_f8_block_plan("bf16", 16, 4096, 4096, 0)["tile_rows"] == 16
    big = dg.gemm_f8_block_plan("bf16", 4096, 4096, 4096, 0)
    assert big == {"tile_rows": 256, "tile_cols": 256, "splits": 1, "workspace_bytes": 0}
    # fp32 sums have the small tile only
    assert dg.gemm_f8_block_plan("f32", 4096, 4096, 4096, 0)["tile_rows"] == 128
    assert dg.gemm_f8_block_plan("bf16", 4096, 4096, 4096, 0, rows_b=1)["tile_rows"] == 256
    deep = dg.gemm_f8_block_plan("bf16", 256, 256, 65536, 1 << 30)
    assert deep["splits"] > 1 and deep["workspace_bytes"] == deep["splits"] * 256 * 256 * 4
    assert dg.gemm_f8_block_plan("bf16", 256, 256, 65536, deep["workspace_bytes"] - 1)["splits"] < deep["splits"]
    with pytest.raises(dg.DgemmError):
        dg.gemm_f8_block_plan("bf16", 64, 64, 64, 0, rows_b=3)
    assert dg.layernorm_bwd_workspace(16384, 4096) == 2 * dg.rmsnorm_bwd_workspace(16384, 4096)
    assert dg.layernorm_bwd_workspace(0, 64) == 0
    with pytest.raises(dg.DgemmError):
        dg.layernorm_bwd_workspace(4, 16385)


FORMS = {"layer_norm": "X weight bias residual f8 keep eps",
         "layer_norm_backward": "dY total weight mean rstd dtotal bias",
         "matmul_f8_block": "A B scale_a scale_b bias act residual out_dtype",
         "quantize_f8_block": "X rows transpose"}


@pytest.mark.parametrize("name", list(FORMS))
def test_signatures_and_host_tensors(name):
    fn = getattr(dg, name)
    assert list(inspect.signature(fn).parameters) == FORMS[name].split() + ["stream"]
    assert fn.__name__ == name and fn.__doc__
    x, w, s = torch.ones(4, 16), torch.ones(16), torch.ones(4, 1)
    kw = {"layer_norm": dict(X=x, weight=w), "layer_norm_backward": dict(dY=x, total=x, weight=w, mean=w[:4], rstd=w[:4]),
          "matmul_f8_block": dict(A=x.to(F8), B=x.to(F8), scale_a=s, scale_b=s),
          "quantize_f8_block": dict(X=x)}[name]
    with pytest.raises(ValueError, match="device tensor"):
        fn(**kw)
    with pytest.raises(ValueError):
        dg.quantize_f8_block(x, rows=64)
    with pytest.raises(ValueError):
        dg.layer_norm(x, w, f8="column")


def test_plain_layer_norm_against_autograd():
    g = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(5, 33, dtype=torch.float64, generator=g) for _ in range(2))
    w, b = (torch.randn(33, dtype=torch.float64, generator=g).requires_grad_() for _ in range(2))
    x.requires_grad_()
    y = torch.nn.functional.layer_norm(x, (33,), w, b, eps=1e-5)
    dx, dw, db = torch.autograd.grad(y, (x, w, b), dy)
    (_, _), (mean, _), (rstd, _), (got, _) = layer64(x.detach(), None, w.detach(), b.detach(), 1e-5)
    assert torch.allclose(got, y.detach(), rtol=1e-12, atol=1e-12)
    (ex, _), (ew, _), (eb, _) = layer_grad64(dy, x.detach(), w.detach(), mean, rstd, None)
    assert torch.allclose(ex, dx, rtol=1e-10, atol=1e-12) and torch.allclose(ew, dw, rtol=1e-10, atol=1e-12)
    assert torch.allclose(eb, db, rtol=1e-12, atol=1e-12)


def test_plain_quantizer_against_torch():
    x = torch.randn(50, 300, generator=torch.Generator().manual_seed(1)).bfloat16()
    q, s = quant_block64(x, 1)
    v = x.double() / s.double().repeat_interleave(128, 1)[:, :300]
    # torch rounds through fp32, whose quotient may lie on the border between two codes where the exact one does not:
    # either code is then within half a step of it
    through = v.float().to(F8).double()
    moved = q != through
    assert moved.float().mean() < 0.01
    assert torch.equal((q - v.float().double()).abs()[moved], (through - v.float().double()).abs()[moved])
    assert ((q - v).abs() <= (through - v).abs()).all()
    q, s = quant_block64(torch.zeros(3, 4), 128)
    assert torch.equal(q, torch.zeros(3, 4, dtype=torch.float64)) and float(s) == 2.0 ** -100


# ------------------------------------------------------------------ gated projections

def gated_call(in_=1, out=1, M=8, N=8, K=8, A=PA, lda=64, Bg=PB, ldbg=64, Bu=PB + 4096, ldbu=64, C=PC, ldc=64, bg=None,
               bu=None, act=4, G=None, ldg=64, U=None, ldu=64, ws=None, ws_bytes=0):
    return lib.gemm_gated(in_, out, M, N, K, V(A), lda, V(Bg), ldbg, V(Bu), ldbu, V(C), ldc, V(bg), V(bu), act, V(G),
                          ldg, V(U), ldu, V(ws), ws_bytes, None)


@pytest.mark.parametrize("want, kw", [
    (INVALID, dict(in_=3)), (INVALID, dict(in_=4)), (INVALID, dict(out=2)), (INVALID, dict(act=5)),
    (INVALID, dict(M=-1)), (INVALID, dict(A=0)), (INVALID, dict(Bg=0)), (INVALID, dict(Bu=0)), (INVALID, dict(C=0)),
    (INVALID, dict(ws_bytes=64)), (LEADING, dict(ldbu=4)), (LEADING, dict(ldbg=4)), (LEADING, dict(G=PZ, ldg=4)),
    (LEADING, dict(U=PZ, ldu=4)), (MISALIGNED, dict(Bu=PB + 4098)), (MISALIGNED, dict(ldbu=65)),
    (MISALIGNED, dict(G=PZ + 2)), (MISALIGNED, dict(bu=PR + 2)), (MISALIGNED, dict(bg=PR + 1)),
    (LARGE, dict(ldbu=1 << 22)), (LARGE, dict(U=FAR, ldu=1 << 22)), (ALIAS, dict(C=PA)), (ALIAS, dict(C=PB + 4096)),
    (ALIAS, dict(G=PC)), (ALIAS, dict(U=PC + 128)), (ALIAS, dict(G=PZ, U=PZ)), (ALIAS, dict(U=PA)), (ALIAS, dict(bu=PC)),
    (ALIAS, dict(M=64, N=64, K=16384, lda=16384, C=FAR, ws=FAR, ws_bytes=1 << 40, Bu=3 * FAR, Bg=4 * FAR, A=5 * FAR)),
])
def test_gemm_gated_refusals(want, kw):
    assert gated_call(**kw) == want


def test_gemm_gated_accepts_until_the_device():
    without_gpu()
    for kw in (dict(), dict(Bu=PB), dict(ldbu=72), dict(Bu=PB + 16, N=8, ldbg=64), dict(G=PZ, U=PZ + 4096, bg=PR, bu=PR),
               dict(G=PZ), dict(U=PZ), dict(K=0, A=0, Bg=0, Bu=0), dict(G=PZ, U=PZ + 32)):
        assert gated_call(**kw) == dg.DGEMM_ERR_DEVICE, kw
    assert gated_call(M=0, A=0, Bg=0, Bu=0, C=0) == dg.DGEMM_OK and gated_call(N=0) == dg.DGEMM_OK


def gated_bwd_call(in_=1, out=1, M=8, N=8, K=8, A=PA, lda=64, Bg=PB, ldbg=64, Bu=PB + 4096, ldbu=64, dC=PC, lddc=64,
                   G=PZ, ldg=64, U=PZ + 4096, ldu=64, act=4, dA=FAR, ldda=64, dBg=2 * FAR, lddbg=64, dBu=3 * FAR,
                   lddbu=64, dbg=None, dbu=None, ws=PW, ws_bytes=1 << 20):
    return lib.gemm_gated_bwd(in_, out, M, N, K, V(A), lda, V(Bg), ldbg, V(Bu), ldbu, V(dC), lddc, V(G), ldg, V(U), ldu,
                              act, V(dA), ldda, V(dBg), lddbg, V(dBu), lddbu, V(dbg), V(dbu), V(ws), ws_bytes, None)


@pytest.mark.parametrize("want, kw", [
    (INVALID, dict(in_=3)), (INVALID, dict(act=9)), (INVALID, dict(K=-1)), (INVALID, dict(G=0)), (INVALID, dict(U=0)),
    (INVALID, dict(dC=0)), (INVALID, dict(A=0)), (INVALID, dict(Bg=0)), (INVALID, dict(Bu=0)), (INVALID, dict(ws=0)),
    (LEADING, dict(lddc=4)), (LEADING, dict(ldg=4)), (LEADING, dict(ldu=4)), (LEADING, dict(ldda=4)),
    (LEADING, dict(lddbg=4)), (LEADING, dict(lddbu=4)), (MISALIGNED, dict(dA=FAR + 8)),
    (MISALIGNED, dict(dbg=PR + 1)), (MISALIGNED, dict(dbu=PR + 2)), (SPACE, dict(ws_bytes=0, ws=0)),
    (SPACE, dict(ws_bytes=64)), (ALIAS, dict(dA=PA)), (ALIAS, dict(dBg=FAR)), (ALIAS, dict(dBu=2 * FAR)),
    (ALIAS, dict(dBu=PZ)), (ALIAS, dict(dbg=PC)), (ALIAS, dict(dbg=PR, dbu=PR)), (ALIAS, dict(ws=PC)),
    (ALIAS, dict(dA=PW)), (LARGE, dict(ldu=1 << 22, U=FAR * 4)),
    (LARGE, dict(in_=0, out=0, M=1 << 21, ws_bytes=1 << 50)),
])
def test_gemm_gated_bwd_refusals(want, kw):
    assert gated_bwd_call(**kw) == want


def test_gemm_gated_bwd_accepts_until_the_device():
    without_gpu()
    for kw in (dict(), dict(dA=None, Bg=0, Bu=0), dict(dBg=None, dBu=None, A=0), dict(dBg=None), dict(U=PZ),
               dict(dbg=PR, dbu=PR + 64), dict(dA=None, dBg=None, dBu=None, A=0, Bg=0, Bu=0, dbg=PR), dict(M=0)):
        assert gated_bwd_call(**kw) == dg.DGEMM_ERR_DEVICE, kw


def test_gated_plans():
    p = dg.gemm_gated_plan("bf16", 8192, 8192, 4096, 0, True)
    assert p == {"tile_rows": 256, "tile_cols": 128, "splits": 1, "workspace_bytes": 0}
    assert dg.gemm_gated_plan("f32", 8192, 8192, 4096, 0)["tile_rows"] == 128
    for M, N, K in [(1, 2048, 8192), (16, 1000, 8200), (64, 500, 4096), (512, 512, 512)]:
        p = dg.gemm_gated_plan("bf16", M, N, K, 1 << 30, True)
        if p["splits"] > 1:
            assert p["workspace_bytes"] == p["splits"] * M * 2 * ((N + 3) // 4 * 4) * 4
            assert dg.gemm_gated_plan("bf16", M, N, K, p["workspace_bytes"] - 1, True)["splits"] < p["splits"]
        assert dg.gemm_gated_plan("bf16", M, N, K, 0, True)["splits"] == 1
    for fmt in ("f32", "bf16", "f16"):
        for M in (1, 16, 100, 3000):
            req, best = dg.gemm_gated_bwd_workspace(fmt, M, 200, 300)
            assert 2 * M * 200 * (4 if fmt == "f32" else 2) < req <= best
    with pytest.raises(dg.DgemmError):
        dg.gemm_gated_plan("f32x3", 8, 8, 8, 0)


def test_gated_signatures_and_host_tensors():
    forms = {"linear_gated": "A Bg Bu bias_g bias_u act out_dtype keep_preact",
             "linear_gated_backward": "A Bg Bu dC gate up act bias"}
    x, w, c = torch.ones(4, 16), torch.ones(16, 8), torch.ones(4, 8)
    for name, params in forms.items():
        fn = getattr(dg, name)
        assert list(inspect.signature(fn).parameters) == params.split() + ["stream"] and fn.__doc__
        with pytest.raises(ValueError, match="device tensor"):
            fn(x, w, w, *((c, c, c) if name.endswith("backward") else ()))
