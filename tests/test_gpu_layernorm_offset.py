"""layernorm of rows whose mean is far from zero: what it loses are half steps of the deviations, not of the mean."""
import pytest
import torch

import dense_gemm_matrix_amd as dg
from tests.feedforward_ref import H, rounded
from tests.linear_ref import padded, sentinel, within

pytestmark = pytest.mark.gpu

EPS = 1e-5
# Additions that a value passes through in a sum: at most 32 columns per thread, 6 steps over a wave's lanes,
# 16 waves.
DEEP = 32 + 6 + 16


def bounds(X, w, b):
    """(mean, rstd, y) in 64 bits and how far they may be off, all roundings being fp32 half steps H: the first
    mean by e0, (DEEP + 2) of them of the row's size; a deviation from it by one of its own; their mean c, which
    takes the place of e0, by ec, DEEP and 3 of the deviations' size; a second subtraction by one more.  The
    variance by DEEP and 6 of the squares' mean, var + e0^2, and by c^2's own error."""
    x = X.double()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    var = d.square().mean(1, keepdim=True)
    rstd = (var + EPS).rsqrt()
    e0 = (DEEP + 2) * H * x.abs().mean(1, keepdim=True)
    ec = (DEEP + 3) * H * (d.abs().mean(1, keepdim=True) + e0)
    ed = H * (d.abs() + e0) + ec + 2 * H * (d.abs() + ec)
    ev = (DEEP + 6) * H * (var + e0.square()) + 2 * e0 * ec + 3 * H * e0.square()
    er = 1.1 * ev / (2 * (var + EPS)) + 6 * H
    y = d * rstd * w.double() + b.double()
    ey = w.double().abs() * rstd * (ed * (1 + er) + d.abs() * er) + 4 * H * (d * rstd * w.double()).abs() + H * y.abs()
    return (mean[:, 0], (ec + H * mean.abs())[:, 0]), (rstd[:, 0], (er * rstd)[:, 0]), (y, ey)


def check(X, dt, seed):
    M, N = X.shape
    g = torch.Generator().manual_seed(seed)
    w, b = 1.0 + 0.2 * torch.randn(N, generator=g), 0.1 * torch.randn(N, generator=g)
    Y, m, r = sentinel(M, N, dt), torch.full((M,), 9.0, device="cuda"), torch.full((M,), 9.0, device="cuda")
    dg.layernorm(padded(X, dt), w.cuda(), b.cuda(), Y, mean=m, rstd=r, eps=EPS)
    torch.cuda.synchronize()
    (mean, em), (rstd, er), (y, ey) = bounds(X, w, b)
    within(m, mean, em)
    within(r, rstd, er)
    within(Y, y, rounded(ey, y, dt))


SIZES = [(5, 7), (9, 128), (3, 250), (4, 500), (3, 1000), (3, 2048), (3, 4096), (300, 4095), (3, 8192), (300, 8190),
         (2, 16384), (2, 32768)]


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("offset", [1e3, -3e4, 1e6])
def test_rows_far_from_zero(size, offset):
    g = torch.Generator().manual_seed(size[1])
    check(torch.randn(*size, generator=g) + offset, torch.float32, 1)


@pytest.mark.parametrize("dt, offset", [(torch.bfloat16, 1e4), (torch.float16, -6e3)], ids=str)
@pytest.mark.parametrize("size", SIZES[::3], ids=lambda s: "x".join(map(str, s)))
def test_16_bit_rows_far_from_zero(dt, offset, size):
    g = torch.Generator().manual_seed(size[1])
    check((100 * torch.randn(*size, generator=g) + offset).to(dt), dt, 2)


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_rows_of_one_value(size):
    """No deviation at all: the reciprocal root is eps', and Y the bias."""
    M, N = size
    check((torch.arange(M)[:, None] * 1234.567 - 321.0).expand(M, N).contiguous(), torch.float32, 3)
