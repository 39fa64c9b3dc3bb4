"""Long batches in fp32: only the transposed copy of A, which dB's product reads, limits
the rows (its row pitch: 256 rows of it stay below 2 GiB)."""
import pytest
import torch

import dense_gemm_matrix_amd as dg
from tests.test_linear_cpu import FAR, bwd_call

LIMIT = 1 << 21
LONG = dict(in_=0, out=0, N=4, K=4, lda=4, ldb=4, lddc=4, ldz=4, ldda=4, lddb=4, A=FAR, dC=2 * FAR, Z=3 * FAR,
            dA=4 * FAR, dB=5 * FAR, ws=6 * FAR, ws_bytes=1 << 32)


@pytest.mark.parametrize("fmt", [0, 3])
def test_only_db_is_limited(fmt):
    kw = dict(LONG, in_=fmt)
    reached = dg.DGEMM_ERR_DEVICE
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU: the pointers are made up")
    assert bwd_call(**dict(kw, M=LIMIT)) == dg.DGEMM_ERR_TOO_LARGE
    assert bwd_call(**dict(kw, M=LIMIT - 3)) == dg.DGEMM_ERR_TOO_LARGE  # a pitch of 4's multiples
    assert bwd_call(**dict(kw, M=LIMIT - 4)) == reached
    for m in (LIMIT, 10 * LIMIT):
        assert bwd_call(**dict(kw, M=m, dB=0, ws_bytes=1 << 36)) == reached
        assert bwd_call(**dict(kw, M=m, dA=0, dB=0, dbias=0x100, ws_bytes=1 << 36)) == reached
        assert bwd_call(**dict(kw, in_=1, out=1, M=m, lda=8, ldb=8, lddc=8, ldz=8, ldda=8, lddb=8,
                               ws_bytes=1 << 36)) == reached


@pytest.mark.gpu
def test_gradients_of_a_long_batch():
    """dA and dbias of 2^21 + 9 rows: dA's rows are those of a call on them alone (with one
    plan for both: a row's sums do not depend on the other rows), dbias the sum in 64 bits
    within its rows' half steps."""
    M, N, K, act = LIMIT + 9, 24, 16, "silu"
    g = torch.Generator().manual_seed(3)
    dC, Z = torch.randn(M, N, generator=g).cuda(), torch.randn(M, N, generator=g).cuda()
    A, B = torch.empty(M, K, device="cuda"), torch.randn(K, N, generator=g).cuda()
    work = torch.empty(dg.gemm_act_bwd_workspace("f32", M, N, K, act, False)[1], dtype=torch.uint8, device="cuda")
    dA, db = torch.full((M, K), float("nan"), device="cuda"), torch.empty(N, device="cuda")
    dg.dgemm_set_plan_override(dg.DGEMM_PLAN_GRID, 128, 128, 1)
    try:
        dg.gemm_act_bwd(A, B, dC, dA=dA, dbias=db, preact=Z, act=act, workspace=work)
        for at in (0, M // 2, M - 4096):
            some = torch.empty(4096, K, device="cuda")
            dg.gemm_act_bwd(A[at:at + 4096], B, dC[at:at + 4096], dA=some, preact=Z[at:at + 4096], act=act,
                            workspace=work)
            assert torch.equal(dA[at:at + 4096], some), at
    finally:
        dg.dgemm_set_plan_override(dg.DGEMM_PLAN_AUTO)
    with pytest.raises(dg.DgemmError):
        dg.gemm_act_bwd(A, B, dC, dB=torch.empty(K, N, device="cuda"), preact=Z, act=act, workspace=work)
    s = torch.sigmoid(Z.double())
    dZ = dC.double() * (s + Z.double() * s * (1 - s))
    # 64 half steps of |dC| (1 + |Z|) per value, and of the absolute sum: 1040 rows per
    # workgroup in 16 runs of 65, then 16 of them, then 2017 workgroups' in 16 runs, 250
    # additions in a row at most
    bound = (64 * (dC.double().abs() * (1 + Z.double().abs())).sum(0) + 250 * dZ.abs().sum(0)) * 2.0 ** -24
    assert bool(((db.double() - dZ.sum(0)).abs() <= bound).all())
