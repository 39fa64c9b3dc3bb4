"""The quantizer's codes are those of the fp32 quotients over the scales' whole range, for
values at and next to ties."""
import pytest
import torch

import dense_gemm_matrix_amd as dg
from tests.linear_ref import F8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("exponent", [-126, -112, -100, -99, -95, -92, -91, -90, -60, 0, 60, 118, 119])
def test_codes_over_the_range_of_scales(exponent):
    g = torch.Generator().manual_seed(exponent + 200)
    m = torch.rand(64, 1, generator=g) + 1.0  # the rows' maxima
    m[:32] = m[:32].bfloat16().float()
    codes = torch.arange(0x7f, dtype=torch.uint8).view(F8).float()
    ties = (codes[1:] + codes[:-1]) / 2 * (m / 448)
    x = torch.cat([m, ties, torch.rand(64, 801, generator=g) * m, ties * (1 + 2.0 ** -23), ties * (1 - 2.0 ** -23)], 1)
    x = torch.minimum(x, m) * 2.0 ** exponent
    x = x[:, :x.shape[1] // 8 * 8].contiguous()
    scale = (x.abs().amax(1) / torch.tensor(448.0)).clamp_min(2.0 ** -100)
    want = (x / scale[:, None]).clamp(-448, 448).to(F8).float()
    Q, got = dg.quantize_f8(x.cuda())
    assert torch.equal(got.cpu(), scale) and torch.equal(Q.cpu().float(), want)
    Q, got = dg.quantize_f8(x.t().contiguous().cuda(), transpose=True)
    assert torch.equal(got.cpu(), scale) and torch.equal(Q.cpu().float(), want)
