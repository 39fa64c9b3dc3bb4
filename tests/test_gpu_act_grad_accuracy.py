"""The gradients of silu and gelu_tanh, value by value against 64 bits, through dbias of
one row (which sums unrounded fp32 values).

f = s + z s (1 - s) p'(z), s the sigmoid of p.  Half steps below are 2^-24.  s: the
reciprocal (2), the sum before it (1 of at most 2, halved), and exp(-|p|)'s own error (2,
and 1.5 |p| of its argument's rounding, where |p| exp(-|p|) <= 0.37) by a slope of at most
1/4: at most 3.4.  The second term is at most 0.36 in size: its factors' errors, about 12
together, are at most 4.3, and exp's argument's part falls with it.  One rounding of the sum,
at most 1.13: 8.9 in all, of 1, where s (1 - s) formed from a rounded s near 1 would be off
by z p'(z), up to 33, half steps."""
import pytest
import torch

import dense_gemm_matrix_amd as dg
from tests.linear_ref import act_grad64

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def gradient(z, act, dt):
    n = len(z)
    _, _, db = dg.linear_backward(torch.ones(1, 8, device="cuda", dtype=dt), torch.ones(8, n, device="cuda", dtype=dt),
                                  torch.ones(1, n, device="cuda", dtype=dt), preact=z[None].cuda(), act=act, bias=True)
    return db.cpu().double()


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("fmt", list(DT))
@pytest.mark.parametrize("lo, hi", [(-30.0, -8.0), (-8.0, -4.0), (-4.0, -1.0), (-1.0, 1.0), (1.0, 2.0), (2.0, 4.0),
                                    (4.0, 8.0), (8.0, 20.0), (20.0, 12000.0)])
def test_gradient_of_one(lo, hi, fmt, act):
    z = torch.linspace(lo, hi, 80000).to(DT[fmt])
    err = (gradient(z, act, DT[fmt]) - act_grad64(z.double(), act)).abs()
    assert float(err.max()) <= 8.9 * 2.0 ** -24, (float(err.max()) * 2 ** 24, float(z[err.argmax()]))


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_far_out_and_nan(act):
    inf, nan = float("inf"), float("nan")
    z = torch.tensor([-inf, -3e38, -1e4, -9e3, -200.0, 200.0, 9e3, 1e4, 3e38, inf, nan, 0.0])
    got = gradient(z, act, torch.float32)
    want = torch.tensor([0.0] * 5 + [1.0] * 5 + [nan, 0.5], dtype=torch.float64)
    assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))
