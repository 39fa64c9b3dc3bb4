"""gelu and its gradient with fp32 outputs, value by value against 64 bits.

Half steps below are 2^-24.  The integral Phi: for |z| < 1, 1/2 + z P(z^2) is off by the
last sum's rounding (half a step of a value below 1) and by z P's few roundings on a value
below 0.35, together at most 1.6 half steps; beyond, exp2 (2 half steps, its argument's
correction under 1), reciprocal (2 and the sum's 1), Q's (1) and three products' roundings, and
the fit (0.25): at most 10.3 half steps of Phi(-|z|) <= 0.159, and for z > 0 the rounding of
1 - Phi(-z) (1): at most 2.7.  gelu = z Phi rounds once more (1 half step of a value of at
most |z|)."""
import math

import pytest
import torch

import dense_gemm_matrix_amd as dg
from tests.linear_ref import act64, act_grad64

pytestmark = pytest.mark.gpu

HS = 2.0 ** -24
# to where exp(-z^2 / 2) leaves fp32's normal range
RANGES = [(-13.0, -8.0), (-8.0, -4.0), (-4.0, -2.0), (-2.0, -1.0), (-1.0, -0.1), (-0.1, 0.1), (0.1, 1.0), (1.0, 4.0),
          (4.0, 60.0)]


def points(lo, hi):
    z = torch.linspace(lo, hi, 100000)
    return torch.cat([z, z * 1e-3, z * 1e-6]) if lo < 0 < hi else z


def check(got, z, ref, slack):
    err = (got.cpu().double() - ref).abs()
    near = 3.7 * HS * z.abs() if slack is None else slack
    worst = (err / near).max()
    assert bool((err <= near).all()), f"{float(worst):.3g} x the bound at {float(z[(err / near).argmax()])}"


@pytest.mark.parametrize("rows", [1, 20, 200], ids=["few rows", "slice", "grid"])
@pytest.mark.parametrize("lo, hi", RANGES)
def test_gelu_fp32(lo, hi, rows):
    if rows == 200:  # a forced grid tile
        dg.dgemm_set_plan_override(dg.DGEMM_PLAN_GRID, 128, 128, 1)
    try:
        z = points(lo, hi)
        z = z[:len(z) // 4 * 4]
        C = dg.linear(torch.ones(rows, 4, device="cuda"),
                      torch.cat([z[None], torch.zeros(3, len(z))]).cuda(), act="gelu")
    finally:
        dg.dgemm_set_plan_override(dg.DGEMM_PLAN_AUTO)
    assert torch.equal(C, C[:1].expand_as(C))
    z64 = z.double()
    ref = act64(z64, "gelu")
    check(C[0], z64, ref, None)
    if hi <= -1:  # relative: the tail's 10.3 half steps and one rounding
        check(C[0], z64, ref, 11.3 * HS * ref.abs())


@pytest.mark.parametrize("lo, hi", RANGES)
def test_gelu_gradient_fp32(lo, hi):
    """Phi + z phi: Phi's 2.7 half steps at most; z phi, at most 0.242 in size where it is
    off the most, within 8 half steps (the exponential's 3, three products, the constant);
    the sum, at most 1.13, one rounding: together at most 5.7 of 1.  On the negative tail
    from -2 on no cancellation is left (|z| phi > 4.7 Phi): 20 half steps relative."""
    z = points(lo, hi)
    z = z[:len(z) // 4 * 4]
    _, _, db = dg.linear_backward(torch.ones(1, 4, device="cuda"), torch.ones(4, len(z), device="cuda"),
                                  torch.ones(1, len(z), device="cuda"), preact=z[None].cuda(), act="gelu", bias=True)
    z64 = z.double()
    ref = act_grad64(z64, "gelu")
    check(db, z64, ref, torch.full_like(z64, 5.7 * HS))
    if hi <= -2:
        check(db, z64, ref, 20 * HS * ref.abs())


def test_fp32_outputs_of_16_bit_operands():
    """The form goes by the output's format: z = 0.03 a, a an integer that both formats hold."""
    a = torch.arange(-200, 201, dtype=torch.float32)
    for dt in (torch.bfloat16, torch.float16):
        w = torch.tensor([[0.03125]]).to(dt)
        A = torch.zeros(20, 8, dtype=dt)
        A[:, 0] = w[0, 0]
        B = torch.zeros(8, 408, dtype=dt)
        B[0, :401] = a.to(dt)
        C = dg.linear(A.cuda(), B.cuda()[:, :408], act="gelu", out_dtype=torch.float32)[0, :401]
        z64 = a.double() * 0.03125
        check(C, z64, act64(z64, "gelu"), (3.7 * HS * z64.abs()).clamp_min(1e-300))


def test_far_out():
    z = torch.tensor([-1e30, -100.0, -20.0, -14.0, 14.0, 20.0, 100.0, 1e30, 3e38])
    C = dg.linear(torch.ones(1, 1, device="cuda"), z[None].cuda(), act="gelu")[0].cpu()
    assert torch.equal(C, torch.where(z > 0, z, torch.zeros_like(z)))
    assert math.isnan(dg.linear(torch.ones(1, 1, device="cuda"), torch.full((1, 4), float("nan"), device="cuda"),
                                act="gelu")[0, 0])
