"""The K split of products of at most 16 rows: a rule on ranges of sizes, and the
products of the plans it chooses."""
import pytest
import torch

import dense_gemm_matrix_amd as dg
from tests.test_gpu_linear import run_act

WS = 1 << 30
KS = [64, 500, 1000, 1024, 1500, 1536, 2000, 2040, 2048, 2056, 2500, 3500, 4000, 4088, 4095, 4096, 4097, 4104, 5120,
      6000, 8184, 8192, 8200, 11008, 14336, 16380, 16384, 20000]
NS = [1, 40, 100, 511, 512, 1000, 2047, 2048, 2880, 4000, 4088, 4095, 4096, 4097, 5000, 5120, 6144, 8184, 8191, 8192,
      8193, 9216, 11008, 12288, 14336, 20000, 28672]


def plan(fmt, M, N, K):
    return dg.gemm_act_plan(fmt, M, N, K, WS, fmt != "f32")


@pytest.mark.parametrize("fmt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M", [1, 16])
def test_split_by_thresholds(fmt, M):
    """Where K is split at one size, it is at every larger K and every smaller N:
    no size is a case of its own."""
    split = {(N, K): plan(fmt, M, N, K)["splits"] > 1 for N in NS for K in KS}
    for N in NS:
        along = [split[N, K] for K in KS]
        assert along == sorted(along), (N, along)
    for K in KS:
        along = [split[N, K] for N in NS]
        assert along == sorted(along, reverse=True), (K, along)


@pytest.mark.parametrize("fmt", ["bf16", "f16", "f32"])
def test_neighbouring_sizes_have_like_plans(fmt):
    """A few columns or terms more or less (the thresholds themselves aside) change
    neither whether K is split nor the workgroups by much.  A threshold among these
    sizes: two pieces of fp32's strips of 64 columns fit 256 workgroups up to
    N = 8192 (128 strips), not beyond."""
    def wgs(N, K):
        p = plan(fmt, 1, N, K)
        return p["splits"] > 1, -(-N // p["tile_cols"]) * p["splits"]
    fits = lambda N: fmt != "f32" or 2 * -(-N // 64) <= 256  # noqa: E731
    for N in (4088, 4096, 8184, 8192, 2048, 1000):
        for K in (4088, 4096, 8192, 16384):
            at = wgs(N, K)
            for n, k in ((N - 7, K), (N + 5, K), (N, K - 8), (N, K + 8), (N, K + 1)):
                near = wgs(n, k)
                if fits(n) != fits(N):
                    assert not near[0]
                    continue
                assert near[0] == at[0] and abs(near[1] - at[1]) <= max(16, at[1] // 4), (N, K, n, k, at, near)


def test_pieces_cover_k_and_fit():
    """At most 16 pieces and 256 workgroups, each piece with k to add."""
    for fmt in ("bf16", "f32"):
        for N in NS:
            for K in KS:
                p = plan(fmt, 4, N, K)
                assert p["tile_rows"] == 16 and 1 <= p["splits"] <= 16
                if p["splits"] > 1:
                    assert -(-N // p["tile_cols"]) * p["splits"] <= 256
                    assert p["workspace_bytes"] == p["splits"] * 4 * ((N + 3) // 4 * 4) * 4
                    assert dg.gemm_act_plan(fmt, 4, N, K, p["workspace_bytes"] - 1, fmt != "f32")["splits"] == 1


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1, 2048), (16, 40, 2050), (3, 700, 2051), (1, 2881, 4088), (16, 4095, 2500),
                                   (5, 5121, 3001), (2, 9000, 3700), (1, 257, 16383)],
                         ids=lambda s: "x".join(map(str, s)))
def test_split_products(fmt, shape):
    M, N, K = shape
    assert plan(fmt, M, N, K)["splits"] > 1 or (fmt == "f32" and N == 9000)
    run_act(fmt, "same", M, N, K, "silu", seed=M + N, ws_bytes=4 << 20)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "f32"])
def test_wide_unsplit_products(fmt):
    """More strips of 32 columns than CUs: strips of 64."""
    assert plan(fmt, 3, 8200, 100)["tile_cols"] == 64 and plan(fmt, 3, 8192, 100)["tile_cols"] == 32
    run_act(fmt, "same", 3, 8200, 100, "gelu_tanh", seed=5)
    run_act(fmt, "same", 16, 8191, 70, "none", seed=6)
