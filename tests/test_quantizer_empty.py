"""Rows (columns, with transpose) without elements: their scale is written all the same,
so that a product over no terms is its bias."""
import ctypes

import pytest
import torch

import dense_gemm_matrix_amd as dg

V = ctypes.c_void_p


@pytest.mark.parametrize("transpose, M, N", [(0, 4, 0), (1, 0, 4)])
def test_a_scale_is_required(transpose, M, N):
    lib = dg.raw()
    assert lib.quant_f8(1, transpose, M, N, V(0), 16, V(0), 16, V(0), None) == dg.DGEMM_ERR_INVALID_VALUE
    assert lib.quant_f8(1, transpose, N, M, V(0), 16, V(0), 16, V(0), None) == dg.DGEMM_OK  # no rows: nothing


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("rows", [1, 3, 70, 1000])
def test_scales_of_empty_rows(dt, rows):
    for shape, tr in (((rows, 0), False), ((0, rows), True)):
        Q = torch.empty(rows, 0, dtype=dg._linear.F8, device="cuda")
        scale = torch.full((rows + 2,), 3.0, device="cuda")
        dg.quant_f8(torch.empty(*shape, dtype=dt, device="cuda"), Q, scale[1:-1], transpose=tr)
        assert bool((scale[1:-1] == 2.0 ** -100).all()) and bool((scale[[0, -1]] == 3.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [2, 40])
def test_product_over_no_terms(rows):
    X, W = torch.empty(rows, 0, device="cuda"), torch.empty(0, 24, device="cuda")
    bias = torch.linspace(-1, 1, 24, device="cuda")
    (A, sa), (B, sb) = dg.quantize_f8(X), dg.quantize_f8(W, transpose=True)
    C = dg.matmul_f8(A, B, sa, sb, bias=bias, out_dtype=torch.float32)
    assert torch.equal(C, bias.expand(rows, 24))
