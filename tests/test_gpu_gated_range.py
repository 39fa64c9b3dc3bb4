"""What a 16-bit gated layer's backward pass does where dG and dU leave the format's range."""
import pytest
import torch

import dense_gemm_matrix_amd as dg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [4, 40, 300])
def test_fp16_products_beyond_the_range(M):
    """dG = dC U = 90000 in one place and 2^-26 in another: infinite and zero to the products in fp16, so in the row
    of dA and the column of dBg that they feed; the biases' sums, and every other row and column, are finite.  In
    bf16 all is finite."""
    N, K = 64, 48
    for dt in (torch.float16, torch.bfloat16):
        one = lambda *s: torch.ones(*s, device="cuda", dtype=dt)  # noqa: E731
        dC, G, U = torch.zeros(M, N, device="cuda", dtype=dt), one(M, N), one(M, N)
        dC[2, 5], U[2, 5], G[2, 5] = 300, 300, 0
        dC[3, 7], U[3, 7], G[3, 7] = 2.0 ** -13, 2.0 ** -13, 0
        dA, dBg, dBu, dbg, dbu = dg.linear_gated_backward(one(M, K), one(K, N), one(K, N), dC, G, U, act="none", bias=True)
        assert float(dbg[5]) == 90000 and float(dbg[7]) == 2.0 ** -26 and (dbu == 0).all() and (dBu == 0).all()
        rest_a, rest_b = torch.arange(M) != 2, torch.arange(N) != 5
        if dt is torch.float16:
            assert dA[2].isinf().all() and dBg[:, 5].isinf().all()
            assert (dA[3] == 0).all() and (dBg[:, 7] == 0).all()
        else:
            assert (dA[2] == 90112).all() and (dBg[:, 5] == 90112).all()  # bf16's nearest to 90000
            assert (dA[3] == 2.0 ** -26).all() and (dBg[:, 7] == 2.0 ** -26).all()
        assert dA[rest_a].isfinite().all() and dBg[:, rest_b].isfinite().all()
