"""The linear layer's entry points on the CPU: refusals come before any device
call, plans are reported without a GPU, and the plain forms the GPU tests use
agree with autograd and with differences."""
import ctypes

import pytest
import torch

import dense_gemm_matrix_amd as dg
from tests.linear_ref import F8, act64, act_grad64, quant64

V = ctypes.c_void_p
PA, PB, PC, PR, PZ, PW = (0x10000000 * i for i in range(1, 7))
FAR = 0x7000000000
lib = dg.raw()


def act_call(in_=1, out=1, M=8, N=8, K=8, A=PA, lda=64, B=PB, ldb=64, C=PC, ldc=64, bias=None, act=4,
             R=None, ldr=64, Z=None, ldz=64, ws=None, ws_bytes=0):
    return lib.gemm_act(in_, out, M, N, K, V(A), lda, V(B), ldb, V(C), ldc, V(bias), act, V(R), ldr,
                        V(Z), ldz, V(ws), ws_bytes, None)


@pytest.mark.parametrize("want, kw", [
    (dg.DGEMM_ERR_INVALID_VALUE, dict(in_=4)), (dg.DGEMM_ERR_INVALID_VALUE, dict(out=2)),
    (dg.DGEMM_ERR_INVALID_VALUE, dict(act=5)), (dg.DGEMM_ERR_INVALID_VALUE, dict(act=-1)),
    (dg.DGEMM_ERR_INVALID_VALUE, dict(M=-1)), (dg.DGEMM_ERR_INVALID_VALUE, dict(A=0)),
    (dg.DGEMM_ERR_INVALID_VALUE, dict(ws_bytes=64)),
    (dg.DGEMM_ERR_LEADING_DIM, dict(R=PR, ldr=4)), (dg.DGEMM_ERR_LEADING_DIM, dict(Z=PZ, ldz=4)),
    (dg.DGEMM_ERR_MISALIGNED, dict(R=PR + 2)), (dg.DGEMM_ERR_MISALIGNED, dict(Z=PZ, ldz=63)),
    (dg.DGEMM_ERR_MISALIGNED, dict(bias=PR + 2)), (dg.DGEMM_ERR_MISALIGNED, dict(ws=PW + 8, ws_bytes=64)),
    (dg.DGEMM_ERR_TOO_LARGE, dict(R=PR, ldr=1 << 22)), (dg.DGEMM_ERR_TOO_LARGE, dict(Z=FAR, ldz=1 << 22)),
    (dg.DGEMM_ERR_ALIAS, dict(R=PC + 256)), (dg.DGEMM_ERR_ALIAS, dict(R=PC, ldr=72)),
    (dg.DGEMM_ERR_ALIAS, dict(Z=PC)), (dg.DGEMM_ERR_ALIAS, dict(Z=PA)), (dg.DGEMM_ERR_ALIAS, dict(R=PZ, Z=PZ)),
    (dg.DGEMM_ERR_ALIAS, dict(bias=PC)), (dg.DGEMM_ERR_ALIAS, dict(C=PA)),
    # a split plan's workspace
    (dg.DGEMM_ERR_ALIAS, dict(M=512, N=4096, K=4096, lda=4096, ldb=4096, ldc=4096, B=FAR, C=2 * FAR, ws=FAR,
                              ws_bytes=1 << 40)),
])
def test_gemm_act_refusals(want, kw):
    assert act_call(**kw) == want


def test_gemm_act_accepts_until_the_device():
    """Valid calls get as far as the device check, also with R in place."""
    want = (dg.DGEMM_ERR_DEVICE,) if not torch.cuda.is_available() else None
    if want is None:
        pytest.skip("needs a machine without a GPU: the pointers are made up")
    assert act_call() in want
    assert act_call(R=PC) in want
    assert act_call(R=PR, Z=PZ, bias=PW) in want
    assert act_call(M=0) == dg.DGEMM_OK and act_call(N=0) == dg.DGEMM_OK


def bwd_call(in_=1, out=1, M=8, N=8, K=8, A=PA, lda=64, B=PB, ldb=64, dC=PC, lddc=64, Z=PZ, ldz=64, act=4,
             dA=FAR, ldda=64, dB=2 * FAR, lddb=64, dbias=None, ws=PW, ws_bytes=1 << 20):
    return lib.gemm_act_bwd(in_, out, M, N, K, V(A), lda, V(B), ldb, V(dC), lddc, V(Z), ldz, act, V(dA),
                            ldda, V(dB), lddb, V(dbias), V(ws), ws_bytes, None)


@pytest.mark.parametrize("want, kw", [
    (dg.DGEMM_ERR_INVALID_VALUE, dict(in_=7)), (dg.DGEMM_ERR_INVALID_VALUE, dict(act=9)),
    (dg.DGEMM_ERR_INVALID_VALUE, dict(K=-1)), (dg.DGEMM_ERR_INVALID_VALUE, dict(Z=0)),
    (dg.DGEMM_ERR_INVALID_VALUE, dict(dC=0)), (dg.DGEMM_ERR_INVALID_VALUE, dict(A=0)),
    (dg.DGEMM_ERR_INVALID_VALUE, dict(B=0)), (dg.DGEMM_ERR_INVALID_VALUE, dict(ws=0)),
    (dg.DGEMM_ERR_LEADING_DIM, dict(lddc=4)), (dg.DGEMM_ERR_LEADING_DIM, dict(ldda=4)),
    (dg.DGEMM_ERR_LEADING_DIM, dict(lddb=4)), (dg.DGEMM_ERR_LEADING_DIM, dict(ldz=4)),
    (dg.DGEMM_ERR_MISALIGNED, dict(dA=FAR + 8)), (dg.DGEMM_ERR_MISALIGNED, dict(dbias=PR + 1)),
    (dg.DGEMM_ERR_WORKSPACE, dict(ws_bytes=0, ws=0)), (dg.DGEMM_ERR_WORKSPACE, dict(ws_bytes=64)),
    (dg.DGEMM_ERR_ALIAS, dict(dA=PA)), (dg.DGEMM_ERR_ALIAS, dict(dB=FAR)), (dg.DGEMM_ERR_ALIAS, dict(dB=PZ)),
    (dg.DGEMM_ERR_ALIAS, dict(dbias=PC)), (dg.DGEMM_ERR_ALIAS, dict(ws=PC)), (dg.DGEMM_ERR_ALIAS, dict(dA=PW)),
    (dg.DGEMM_ERR_TOO_LARGE, dict(ldz=1 << 22, dC=FAR * 3, Z=FAR * 4)),
])
def test_gemm_act_bwd_refusals(want, kw):
    assert bwd_call(**kw) == want


def f8_call(out=1, M=8, N=8, K=8, A=PA, lda=64, B=PB, ldb=64, C=PC, ldc=64, sa=PR, sb=PR + 256, bias=None,
            act=0, R=None, ldr=64, ws=None, ws_bytes=0):
    return lib.gemm_f8(out, M, N, K, V(A), lda, V(B), ldb, V(C), ldc, V(sa), V(sb), V(bias), act, V(R), ldr,
                       V(ws), ws_bytes, None)


@pytest.mark.parametrize("want, kw", [
    (dg.DGEMM_ERR_INVALID_VALUE, dict(out=3)), (dg.DGEMM_ERR_INVALID_VALUE, dict(act=5)),
    (dg.DGEMM_ERR_INVALID_VALUE, dict(N=-1)), (dg.DGEMM_ERR_INVALID_VALUE, dict(sa=0)),
    (dg.DGEMM_ERR_INVALID_VALUE, dict(sb=0)), (dg.DGEMM_ERR_INVALID_VALUE, dict(B=0)),
    (dg.DGEMM_ERR_LEADING_DIM, dict(lda=0)), (dg.DGEMM_ERR_LEADING_DIM, dict(K=80)),
    (dg.DGEMM_ERR_MISALIGNED, dict(lda=72)), (dg.DGEMM_ERR_MISALIGNED, dict(B=PB + 8)),
    (dg.DGEMM_ERR_MISALIGNED, dict(sa=PR + 2)), (dg.DGEMM_ERR_TOO_LARGE, dict(lda=1 << 23)),
    (dg.DGEMM_ERR_ALIAS, dict(C=PA)), (dg.DGEMM_ERR_ALIAS, dict(C=PB)), (dg.DGEMM_ERR_ALIAS, dict(sa=PC)),
    (dg.DGEMM_ERR_ALIAS, dict(R=PC + 128)),
])
def test_gemm_f8_refusals(want, kw):
    assert f8_call(**kw) == want


def norm_call(in_=1, out=0, M=4, N=64, X=PA, ldx=64, R=None, ldr=64, S=None, lds=64, w=PW, eps=1e-6, Y=PC,
              ldy=64, scale=None, rstd=None):
    return lib.rmsnorm(in_, out, M, N, V(X), ldx, V(R), ldr, V(S), lds, V(w), eps, V(Y), ldy, V(scale),
                       V(rstd), None)


@pytest.mark.parametrize("want, kw", [
    (dg.DGEMM_ERR_INVALID_VALUE, dict(in_=3)), (dg.DGEMM_ERR_INVALID_VALUE, dict(out=2)),
    (dg.DGEMM_ERR_INVALID_VALUE, dict(w=0)), (dg.DGEMM_ERR_INVALID_VALUE, dict(eps=-1.0)),
    (dg.DGEMM_ERR_INVALID_VALUE, dict(eps=float("nan"))), (dg.DGEMM_ERR_INVALID_VALUE, dict(out=1)),
    (dg.DGEMM_ERR_INVALID_VALUE, dict(scale=PR)), (dg.DGEMM_ERR_INVALID_VALUE, dict(Y=0)),
    (dg.DGEMM_ERR_LEADING_DIM, dict(ldx=56)), (dg.DGEMM_ERR_MISALIGNED, dict(w=PW + 4)),
    (dg.DGEMM_ERR_MISALIGNED, dict(Y=PC + 8)), (dg.DGEMM_ERR_MISALIGNED, dict(rstd=PR + 2)),
    (dg.DGEMM_ERR_TOO_LARGE, dict(N=32776, ldx=32776, ldy=32776, Y=FAR)),
    (dg.DGEMM_ERR_ALIAS, dict(Y=PA + 128)), (dg.DGEMM_ERR_ALIAS, dict(S=PC)), (dg.DGEMM_ERR_ALIAS, dict(Y=PW)),
    (dg.DGEMM_ERR_ALIAS, dict(out=1, scale=PR, Y=PA)), (dg.DGEMM_ERR_ALIAS, dict(rstd=PA)),
    (dg.DGEMM_ERR_ALIAS, dict(R=PR, Y=PR, ldr=128, ldy=64)),
])
def test_rmsnorm_refusals(want, kw):
    assert norm_call(**kw) == want


def norm_bwd_call(in_=1, M=4, N=64, dY=PA, S=PB, w=PW, rstd=PR, dS=None, dX=PC, lddx=64, dw=None, ws=None,
                  ws_bytes=0, ld=64):
    return lib.rmsnorm_bwd(in_, M, N, V(dY), ld, V(S), ld, V(w), V(rstd), V(dS), ld, V(dX), lddx, V(dw),
                           V(ws), ws_bytes, None)


@pytest.mark.parametrize("want, kw", [
    (dg.DGEMM_ERR_INVALID_VALUE, dict(in_=4)), (dg.DGEMM_ERR_INVALID_VALUE, dict(w=0)),
    (dg.DGEMM_ERR_INVALID_VALUE, dict(rstd=0)), (dg.DGEMM_ERR_INVALID_VALUE, dict(dX=0)),
    (dg.DGEMM_ERR_LEADING_DIM, dict(lddx=8)), (dg.DGEMM_ERR_MISALIGNED, dict(dY=PA + 2)),
    (dg.DGEMM_ERR_WORKSPACE, dict(dw=PZ)), (dg.DGEMM_ERR_WORKSPACE, dict(dw=PZ, ws=FAR, ws_bytes=255)),
    (dg.DGEMM_ERR_TOO_LARGE, dict(N=16392, ld=16392, lddx=16392, S=FAR, dX=2 * FAR)),
    (dg.DGEMM_ERR_ALIAS, dict(dX=PB)), (dg.DGEMM_ERR_ALIAS, dict(dX=PA + 128)),
    (dg.DGEMM_ERR_ALIAS, dict(dw=PA, ws=FAR, ws_bytes=1 << 20)),
])
def test_rmsnorm_bwd_refusals(want, kw):
    assert norm_bwd_call(**kw) == want


@pytest.mark.parametrize("want, kw", [
    (dg.DGEMM_ERR_INVALID_VALUE, dict(in_=3)), (dg.DGEMM_ERR_INVALID_VALUE, dict(tr=2)),
    (dg.DGEMM_ERR_INVALID_VALUE, dict(scale=0)), (dg.DGEMM_ERR_LEADING_DIM, dict(ldq=16)),
    (dg.DGEMM_ERR_LEADING_DIM, dict(tr=1, M=80)), (dg.DGEMM_ERR_MISALIGNED, dict(ldq=72)),
    (dg.DGEMM_ERR_MISALIGNED, dict(Q=PC + 4)), (dg.DGEMM_ERR_ALIAS, dict(Q=PA)),
    (dg.DGEMM_ERR_TOO_LARGE, dict(N=32776, ldx=32776, ldq=32784)),
])
def test_quant_f8_refusals(want, kw):
    a = dict(in_=1, tr=0, M=4, N=64, X=PA, ldx=64, Q=PC, ldq=64, scale=PR)
    a.update(kw)
    assert lib.quant_f8(a["in_"], a["tr"], a["M"], a["N"], V(a["X"]), a["ldx"], V(a["Q"]), a["ldq"],
                        V(a["scale"]), None) == want


def test_workspace_status_string():
    msg = dg.dgemm_status_string(dg.DGEMM_ERR_WORKSPACE)
    assert msg.startswith("DGEMM_ERR_WORKSPACE")


def test_plans():
    p = dg.gemm_act_plan("bf16", 1, 4096, 4096, 0, True)
    assert p["tile_rows"] == 16 and p["splits"] == 1 and p["workspace_bytes"] == 0
    # deep K is split where a workspace allows it
    for M, N, K in [(1, 2048, 8192), (16, 4096, 8192), (1, 1024, 16384), (4, 12288, 8200)]:
        p = dg.gemm_act_plan("bf16", M, N, K, 1 << 30, True)
        assert p["tile_rows"] == 16 and p["splits"] > 1
        assert p["workspace_bytes"] == p["splits"] * M * N * 4
        assert dg.gemm_act_plan("bf16", M, N, K, p["workspace_bytes"] - 1, True)["splits"] == 1
    # above the few-row kernel's 16 rows: gemm_ex's plan, never Stream-K
    assert dg.gemm_act_plan("bf16", 512, 4096, 4096, 0, True) == {
        k: v for k, v in dg.gemm_ex_plan("bf16", 512, 4096, 4096, 0, True).items() if k != "stream_k"}
    assert dg.gemm_f8_plan("bf16", 16, 4096, 4096, 0)["tile_rows"] == 16
    deep = dg.gemm_f8_plan("bf16", 64, 64, 16384, 1 << 30)
    assert deep["splits"] > 1 and deep["workspace_bytes"] == deep["splits"] * 64 * 64 * 4
    assert dg.gemm_f8_plan("bf16", 64, 64, 16384, deep["workspace_bytes"] - 1)["splits"] < deep["splits"]
    assert dg.gemm_f8_plan("bf16", 64, 64, 16384, 0)["splits"] == 1
    for fmt in ("f32", "bf16", "f16", "f32x3"):
        for act in dg.ACT_CODES:
            req, best = dg.gemm_act_bwd_workspace(fmt, 100, 200, 300, act)
            assert 0 < req <= best
            # few rows: no transposes, no partial sums; nothing at all where dC serves as dZ
            few, few_best = dg.gemm_act_bwd_workspace(fmt, 16, 200, 300, act, fmt[:3] != "f32")
            assert few == few_best and (few == 0) == (act == "none")
    assert dg.rmsnorm_bwd_workspace(16384, 4096) >= 4096 * 4
    assert dg.rmsnorm_bwd_workspace(0, 64) == 0
    with pytest.raises(dg.DgemmError):
        dg.rmsnorm_bwd_workspace(4, 16385)


def test_bindings_check_arguments():
    x = torch.zeros(4, 16)
    with pytest.raises(ValueError):
        dg.gemm_act(x, x.t().contiguous(), torch.zeros(4, 4))      # not on a GPU
    with pytest.raises(ValueError):
        dg.rms_norm(x, torch.ones(16))
    with pytest.raises(ValueError):
        dg.quantize_f8(x)
    with pytest.raises(ValueError):
        dg.linear(x[0], x)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_plain_gradient_against_autograd_and_differences(act):
    z = torch.linspace(-9, 9, 1001, dtype=torch.float64) + 1e-3
    t = z.clone().requires_grad_(True)
    (g,) = torch.autograd.grad(act64(t, act).sum(), t)
    assert torch.allclose(act_grad64(z, act), g, rtol=1e-12, atol=1e-13)
    h = 1e-6
    d = (act64(z + h, act) - act64(z - h, act)) / (2 * h)
    # central differences: h^2 / 6 times a third derivative of a few units, and
    # cancellation of 2^-52 |value| / h
    assert torch.allclose(act_grad64(z, act), d, rtol=0, atol=1e-8)


def test_plain_quantizer_against_torch():
    y = torch.randn(50, 70, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    q, s = quant64(y)
    assert torch.equal(q, (y / s[:, None]).float().to(F8).double())
    assert torch.equal(quant64(torch.zeros(1, 4, dtype=torch.float64))[0], torch.zeros(1, 4, dtype=torch.float64))
