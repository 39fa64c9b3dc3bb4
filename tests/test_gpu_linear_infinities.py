"""Infinite pre-activations: every kernel's epilogue gives what the activations'
definitions give (include/dgemm.h), the same as act64's in 64 bits: +infinity at
+infinity for all of them; at -infinity -infinity without an activation, 0 for relu
and, for the others, the NaN of the definition's -inf * 0."""
import pytest
import torch

import dense_gemm_matrix_amd as dg
from tests.linear_ref import F8, act64, padded, sentinel

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
INF = float("inf")
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
# plan: (rows, forced tile and splits); few rows unsplit and split, slice-K, grid, split grid
PLANS = {"few": (1, None), "few-split": (5, (16, 64, 3)), "slice": (20, (32, 32, 4)), "slice64": (40, (64, 64, 4)),
         "grid": (40, (128, 128, 1)), "grid-large": (260, (256, 256, 1)), "split": (40, (128, 128, 3))}


@pytest.fixture
def plan(request):
    rows, tile = PLANS[request.param]
    if tile:
        dg.dgemm_set_plan_override(dg.DGEMM_PLAN_GRID, *tile)
    yield rows
    dg.dgemm_set_plan_override(dg.DGEMM_PLAN_AUTO)


def same(got, want):
    assert torch.equal(torch.nan_to_num(got, 7.0, 9e30, -9e30), torch.nan_to_num(want, 7.0, 9e30, -9e30)), \
        (got[0].tolist(), want[0].tolist())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("fmt", list(DT))
@pytest.mark.parametrize("plan", list(PLANS), indirect=True)
def test_infinite_operands(plan, fmt, act):
    dt, K = DT[fmt], 200
    z = torch.tensor([INF, -INF, 1.0, INF, 0.0, -INF, -2.0, INF])
    B = torch.zeros(K, len(z))
    B[0] = z
    C, Z = sentinel(plan, len(z), dt), sentinel(plan, len(z), dt)
    ws = torch.empty(4 << 20, dtype=torch.uint8, device="cuda")
    dg.gemm_act(padded(torch.ones(plan, K), dt), padded(B, dt), C, act=act, preact=Z, workspace=ws)
    inf = torch.isinf(z)
    same(Z.cpu().float(), z.expand(plan, -1))
    same(C.cpu().float()[:, inf], act64(z.double(), act).float()[inf].expand(plan, -1))
    assert torch.isfinite(C.cpu().float()[:, ~inf]).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("fmt", ["bf16", "f32"])
@pytest.mark.parametrize("plan", list(PLANS), indirect=True)
def test_sums_past_the_largest_value(plan, fmt, act):
    """Finite operands whose fp32 sum overflows."""
    dt, K = DT[fmt], 200
    B = torch.zeros(K, 4)
    B[:, 0], B[:, 1], B[:, 3] = 3e38, -3e38, 1.0
    C = sentinel(plan, 4, dt)
    ws = torch.empty(4 << 20, dtype=torch.uint8, device="cuda")
    dg.gemm_act(padded(torch.ones(plan, K), dt), padded(B, dt), C, act=act, workspace=ws)
    want = act64(torch.tensor([INF, -INF], dtype=torch.float64), act).float()
    same(C.cpu().float()[:, :2], want.expand(plan, -1))
    assert torch.isfinite(C.cpu().float()[:, 2:]).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("od", [torch.float32, torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("plan", [p for p in PLANS if p != "few-split"], indirect=True)
def test_infinite_scales_of_8_bit_products(plan, od, act):
    K = 300
    A, B = torch.ones(plan, K), torch.zeros(6, K)
    B[:, 0] = torch.tensor([2.0, -2.0, 1.0, -1.0, 4.0, 0.5])
    sb = torch.tensor([INF, INF, 1.0, 1.0, INF, 1.0])
    C = sentinel(plan, 6, od)
    ws = torch.empty(4 << 20, dtype=torch.uint8, device="cuda")
    dg.gemm_f8(padded(A, F8), padded(B, F8), C, torch.ones(plan, device="cuda"), sb.cuda(), act=act, workspace=ws)
    want = act64(torch.tensor([INF, -INF, INF], dtype=torch.float64), act).float()
    same(C.cpu().float()[:, [0, 1, 4]], want.expand(plan, -1))
    assert torch.isfinite(C.cpu().float()[:, [2, 3, 5]]).all()


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("fmt", list(DT))
@pytest.mark.parametrize("rows", [1, 40])
def test_gradients_at_infinity(rows, fmt, act):
    """The derivatives' limits: 1 at +infinity, 0 at -infinity; a NaN stays one."""
    dt = DT[fmt]
    Z = torch.tensor([INF, -INF, float("nan"), 1e6, -1e6]).expand(rows, 5)
    _, _, db = dg.linear_backward(padded(torch.ones(rows, 8), dt), padded(torch.ones(8, 5), dt),
                                  padded(torch.ones(rows, 5), dt), preact=padded(Z, dt), act=act, bias=True)
    same(db.cpu()[None], torch.tensor([[rows, 0.0, float("nan"), rows, 0.0]]))
