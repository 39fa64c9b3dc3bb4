"""A plan query's bytes are the bytes its plan takes: asked again with exactly those it answers the same plan,
with fewer another one, and the allocating forms, which allocate what the query says, run the plan it names."""
import random

import pytest
import torch

import dense_gemm_matrix_amd as dg

ANY = 1 << 40


def sizes(seed, count=400):
    """M up to 16, N and K spread over their logarithm, with the depths from which K is split among them."""
    rng = random.Random(seed)
    for _ in range(count):
        yield rng.randint(1, 16), int(2 ** rng.uniform(0, 15)), int(2 ** rng.uniform(10, 15))


def same_with_its_bytes(query, shapes):
    split = 0
    for shape in shapes:
        p = query(*shape, ANY)
        assert query(*shape, p["workspace_bytes"]) == p, shape
        if p["splits"] > 1:
            split += 1
            assert query(*shape, p["workspace_bytes"] - 1)["workspace_bytes"] < p["workspace_bytes"], shape
        else:
            assert p["workspace_bytes"] == 0, shape
    assert split > 20


GATED = [(1, 1024, 4096), (1, 512, 4096), (1, 1024, 5120), (8, 512, 7168), (3, 298, 8002)]


@pytest.mark.parametrize("fmt", ["bf16", "f16", "f32"])
def test_gated_rows_split_with_the_reported_bytes(fmt):
    same_with_its_bytes(lambda M, N, K, ws: dg.gemm_gated_plan(fmt, M, N, K, ws, fmt != "f32"),
                        GATED + list(sizes(1)))


@pytest.mark.parametrize("cols", [32, 64])
def test_forced_gated_strips_take_what_they_report(cols):
    """Few steps of K: pieces of an odd number of steps may leave a single one, which takes no workspace."""
    dg.dgemm_set_plan_override(dg.DGEMM_PLAN_GRID, 16, cols, 2)
    try:
        for K in (32, 64, 96, 100, 128, 160, 4096):
            p = dg.gemm_gated_plan("bf16", 4, 40, K, ANY, True)
            assert (p["workspace_bytes"] > 0) == (p["splits"] > 1), K
            assert dg.gemm_gated_plan("bf16", 4, 40, K, p["workspace_bytes"], True) == p, K
    finally:
        dg.dgemm_set_plan_override(dg.DGEMM_PLAN_AUTO)


ACT = [(1, 1024, 4096), (1, 512, 4096), (2, 336, 11856), (8, 512, 7168), (3, 298, 8002)]


@pytest.mark.parametrize("fmt", ["bf16", "f16", "f32"])
def test_rows_split_with_the_reported_bytes(fmt):
    same_with_its_bytes(lambda M, N, K, ws: dg.gemm_act_plan(fmt, M, N, K, ws, fmt != "f32"), ACT + list(sizes(2)))


@pytest.mark.parametrize("cols", [32, 64, 128])
def test_forced_strips_take_what_they_report(cols):
    dg.dgemm_set_plan_override(dg.DGEMM_PLAN_GRID, 16, cols, 2)
    try:
        for K in (32, 64, 96, 100, 128, 160, 4096):
            p = dg.gemm_act_plan("bf16", 4, 40, K, ANY, True)
            assert (p["workspace_bytes"] > 0) == (p["splits"] > 1), K
            assert dg.gemm_act_plan("bf16", 4, 40, K, p["workspace_bytes"], True) == p, K
    finally:
        dg.dgemm_set_plan_override(dg.DGEMM_PLAN_AUTO)


@pytest.mark.parametrize("M, N, K", [(2 ** 31 - 1, 4096, 64), (2 ** 31 - 1, 8000, 200), (2 ** 30, 8192, 8)])
def test_more_small_tiles_than_a_launch_counts(M, N, K):
    """Outputs with more 64 x 64 tiles than 2^31: a larger tile's plan, not one without a tile."""
    for fmt in ("f32", "bf16", "f16"):
        p = dg.gemm_gated_plan(fmt, M, N, K, 0, fmt != "f32")
        assert p["tile_rows"] >= 64 and p["tile_cols"] >= 32 and p["splits"] == 1
        for rows_b in (1, 128):
            p = dg.gemm_f8_block_plan(fmt, M, N, K, 0, rows_b)
            assert p["tile_rows"] >= 64 and p["splits"] == 1


@pytest.fixture
def no_such_tile():
    """A grid override that no kernel has: the automatic plans."""
    yield lambda t=512: dg.dgemm_set_plan_override(dg.DGEMM_PLAN_GRID, t, t, 1)
    dg.dgemm_set_plan_override(dg.DGEMM_PLAN_AUTO)


@pytest.mark.parametrize("tile", [16, 96, 192, 512, 1024])
@pytest.mark.parametrize("fmt", ["f32", "bf16", "f16"])
def test_gated_backward_under_a_tile_that_no_kernel_has(fmt, tile, no_such_tile):
    shapes = [(8, 4096, 1024), (1000, 2744, 1032), (4096, 578, 488), (300, 1500, 900)]
    auto = [dg.gemm_gated_bwd_workspace(fmt, *x) for x in shapes]
    no_such_tile(tile)
    assert [dg.gemm_gated_bwd_workspace(fmt, *x) for x in shapes] == auto


@pytest.mark.parametrize("fmt", ["f32", "bf16", "f16"])
def test_block_products_under_a_tile_that_no_kernel_has(fmt, no_such_tile):
    """fp32 C has no 256 x 256 tile; a split without its workspace is not a plan, and one of more pieces than
    K has steps is reduced to whole steps (5 steps in 4 pieces: 2, 2 and 1)."""
    shapes = [(300, 1000, 2000), (4096, 4096, 4096), (700, 5000, 3000), (2048, 4096, 8192), (40, 4096, 640)]
    plans = lambda ws: [dg.gemm_f8_block_plan(fmt, *x, ws, r) for x in shapes for r in (1, 128)]  # noqa: E731
    auto = {ws: plans(ws) for ws in (0, ANY)}
    for tile in (16, 192, 512) + ((256,) if fmt == "f32" else ()):
        no_such_tile(tile)
        assert {ws: plans(ws) for ws in (0, ANY)} == auto, tile
    dg.dgemm_set_plan_override(dg.DGEMM_PLAN_GRID, 128, 128, 4)
    assert plans(0) == auto[0]
    for p, (M, N, K) in zip(plans(ANY), [x for x in shapes for _ in (1, 128)]):
        pieces = 3 if K == 640 else 4
        assert p == {"tile_rows": 128, "tile_cols": 128, "splits": pieces, "workspace_bytes": pieces * M * N * 4}


@pytest.mark.gpu
@pytest.mark.parametrize("tile", [192, 512])
@pytest.mark.parametrize("fmt", ["f32", "bf16"])
def test_gated_backward_runs_under_a_tile_that_no_kernel_has(fmt, tile, no_such_tile):
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[fmt]
    gen = torch.Generator(device="cuda").manual_seed(tile)
    M, N, K = 72, 136, 264
    rnd = lambda r, c: torch.randn(r, c, generator=gen, device="cuda").to(dt)  # noqa: E731
    args = rnd(M, K), rnd(K, N), rnd(K, N), rnd(M, N), rnd(M, N), rnd(M, N)
    want = dg.linear_gated_backward(*args, bias=True)
    no_such_tile(tile)
    for got, ref in zip(dg.linear_gated_backward(*args, bias=True), want):
        assert torch.equal(got, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", ACT, ids=lambda s: "x".join(map(str, s)))
def test_rows_with_their_bytes_as_with_more(shape):
    """linear runs the plan that a larger workspace gets: the same bits."""
    M, N, K = shape
    gen = torch.Generator(device="cuda").manual_seed(M + N + K)
    A = torch.randn(M, (K + 7) // 8 * 8, generator=gen, device="cuda").bfloat16()[:, :K]
    B = torch.randn(K, (N + 7) // 8 * 8, generator=gen, device="cuda").bfloat16()[:, :N]
    C = torch.empty(M, (N + 7) // 8 * 8, device="cuda", dtype=torch.bfloat16)[:, :N]
    dg.gemm_act(A, B, C, act="silu", workspace=torch.empty(8 << 20, device="cuda", dtype=torch.uint8))
    assert torch.equal(dg.linear(A, B, act="silu"), C)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", GATED, ids=lambda s: "x".join(map(str, s)))
def test_gated_with_its_bytes_as_with_more(shape):
    """linear_gated runs the plan that a larger workspace gets: the same bits."""
    M, N, K = shape
    gen = torch.Generator(device="cuda").manual_seed(M + N + K)
    A = torch.randn(M, (K + 7) // 8 * 8, generator=gen, device="cuda").bfloat16()[:, :K]
    Bg, Bu = (torch.randn(K, (N + 7) // 8 * 8, generator=gen, device="cuda").bfloat16()[:, :N] for _ in range(2))
    C = torch.empty(M, (N + 7) // 8 * 8, device="cuda", dtype=torch.bfloat16)[:, :N]
    dg.gemm_gated(A, Bg, Bu, C, workspace=torch.empty(8 << 20, device="cuda", dtype=torch.uint8))
    assert torch.equal(dg.linear_gated(A, Bg, Bu), C)
