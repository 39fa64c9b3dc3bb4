"""rmsnorm with a scale per row and block of 128 columns: how many scales the C entry writes, and where, is what
include/dgemm.h says."""
import ctypes
import os
import re

import pytest
import torch

import dense_gemm_matrix_amd as dg

V = ctypes.c_void_p
lib = dg.raw()


def contract():
    """The comment above rmsnorm's declaration, on one line."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "dgemm.h")
    head = open(path).read().split("int rmsnorm(")[0]
    return re.sub(r"\s*\n \* *", " ", head[head.rindex("/*"):])


def test_the_header_names_the_block_scales():
    text = contract()
    assert "DGEMM_ROWS_F8_BLOCK" in text and "M * ceil(N / 128)" in text and "scale[b * M + i]" in text
    assert "DGEMM_ROWS_F8 and only then" not in text


@pytest.mark.parametrize("f8", [None, 0, 1, 2, False, True, "row", "block"])
def test_norms_take_any_truth_value(f8):
    """f8 is a truth value, or names the scales; other names are refused."""
    x, w = torch.ones(4, 16), torch.ones(16)
    for norm in (dg.rms_norm, dg.layer_norm):
        with pytest.raises(ValueError, match="device tensor"):
            norm(x, w, f8=f8)
        for name in ("rows", "e4m3", ""):
            with pytest.raises(ValueError, match="f8 must be"):
                norm(x, w, f8=name)


@pytest.mark.gpu
@pytest.mark.parametrize("f8", [None, 0, 2, True])
def test_truth_values_on_the_device(f8):
    x, w = torch.ones(4, 16, device="cuda"), torch.ones(16, device="cuda")
    assert ("scale" in dg.rms_norm(x, w, f8=f8)) == bool(f8)


@pytest.mark.gpu
@pytest.mark.parametrize("M, N", [(1, 1), (1, 129), (3, 128), (5, 1000), (17, 257), (300, 4096)])
def test_block_scales_where_the_header_says(M, N):
    """Every scale against the same norm's fp32 output, and nothing before or behind them."""
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    ld = (N + 15) // 16 * 16
    X = torch.randn(M, ld, generator=gen, device="cuda")
    w = torch.rand(ld, generator=gen, device="cuda") + 0.5
    Y = torch.empty(M, ld, device="cuda")
    Q = torch.empty(M, ld, device="cuda", dtype=torch.uint8)
    blocks = (N + 127) // 128
    buf = torch.full((64 + M * blocks + 64,), 77.0, device="cuda")
    stream = V(torch.cuda.current_stream().cuda_stream)
    for out, to, scale in ((0, Y, None), (2, Q, buf.data_ptr() + 256)):
        assert lib.rmsnorm(0, out, M, N, V(X.data_ptr()), ld, None, ld, None, ld, V(w.data_ptr()), 1e-6,
                           V(to.data_ptr()), ld, V(scale), None, stream) == dg.DGEMM_OK
    torch.cuda.synchronize()
    assert (buf[:64] == 77).all() and (buf[64 + M * blocks:] == 77).all()
    got = buf[64:64 + M * blocks].view(blocks, M).t().cpu()
    y = torch.zeros(M, blocks * 128)
    y[:, :N] = Y[:, :N].cpu()
    # y's fp32 values are the ones the 8-bit pass divides (one kernel's arithmetic); the scale is their largest
    # by 448, one fp32 quotient.  (Rows of 2049 to 8192 columns in batches up to 256, which the plain output sums in
    # another order, are not among these sizes.)
    want = (y.view(M, blocks, 128).abs().amax(2) / torch.tensor(448.0)).clamp_min(2.0 ** -100)
    assert torch.equal(got, want)
