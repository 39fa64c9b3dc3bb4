"""Binding of a feed-forward block's operators (include/dgemm.h) beside _linear's:
gated projections and layer norms with their gradients, and products of 8-bit
operands with a scale per block of 128.  As there, the functions named like the C entry points (in _marshal)
marshal tensors that the caller has allocated, the others allocate their results
and workspaces, and nothing is recorded for autograd."""
import ctypes

import torch

from ._binding import DGEMM_OUT_F32, DGEMM_OUT_SAME, IN_CODES, _TORCH_IN, _check, _lib, _shapes
from ._linear import (
    F8, F8_BLOCK, _ANY, _block_scales, _blocks, _bytes, _device_tensor, _empty, _formats, _norm_results, _on_stream,
    _plan,
)
from ._marshal import (  # noqa: F401
    gemm_f8_block, gemm_gated, gemm_gated_bwd, layernorm, layernorm_bwd, quant_f8_block,
)

_i, _p, _sz, _f = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
_P, _PS = ctypes.POINTER(_i), ctypes.POINTER(_sz)
_ARGTYPES = {
    "gemm_gated": [_i] * 5 + [_p, _i] * 4 + [_p, _p, _i] + [_p, _i] * 2 + [_p, _sz, _p],
    "gemm_gated_plan": [_i] * 5 + [_sz, _P, _P, _P, _PS],
    "gemm_gated_bwd": [_i] * 5 + [_p, _i] * 6 + [_i] + [_p, _i] * 3 + [_p, _p, _p, _sz, _p],
    "gemm_gated_bwd_workspace": [_i] * 5 + [_PS, _PS],
    "gemm_f8_block": [_i] * 5 + [_p, _i] * 3 + [_p, _i, _i] * 2 + [_p, _i, _p, _i, _p, _sz, _p],
    "gemm_f8_block_plan": [_i] * 5 + [_sz, _P, _P, _P, _PS],
    "quant_f8_block": [_i] * 5 + [_p, _i] * 2 + [_p, _i, _i, _p],
    "layernorm": [_i] * 4 + [_p, _i] * 3 + [_p, _p, _f, _p, _i, _p, _i, _i, _p, _p, _p],
    "layernorm_bwd": [_i] * 3 + [_p, _i] * 2 + [_p] * 3 + [_p, _i] * 2 + [_p, _p, _p, _sz, _p],
    "layernorm_bwd_workspace": [_i, _i, _PS],
}
for _name, _types in _ARGTYPES.items():
    getattr(_lib, _name).argtypes = _types
    getattr(_lib, _name).restype = _i


def gemm_gated_plan(in_fmt: str, M: int, N: int, K: int, workspace_bytes: int, out_same: bool = False) -> dict:
    """Host query of the plan gemm_gated uses with `workspace_bytes` available."""
    return _plan(_lib.gemm_gated_plan, IN_CODES[in_fmt], DGEMM_OUT_SAME if out_same else DGEMM_OUT_F32,
                 M, N, K, int(workspace_bytes))


def gemm_gated_bwd_workspace(in_fmt: str, M: int, N: int, K: int, out_same: bool = True):
    """(required, best) workspace bytes of gemm_gated_bwd."""
    req, best = _sz(0), _sz(0)
    _check(_lib.gemm_gated_bwd_workspace(IN_CODES[in_fmt], DGEMM_OUT_SAME if out_same else DGEMM_OUT_F32, M, N, K,
                                         ctypes.byref(req), ctypes.byref(best)))
    return req.value, best.value


def gemm_f8_block_plan(out_fmt: str, M: int, N: int, K: int, workspace_bytes: int, rows_b: int = F8_BLOCK) -> dict:
    """Host query of the plan gemm_f8_block uses with `workspace_bytes` available; rows_b: rows
    of B that share a scale, 128 or 1."""
    return _plan(_lib.gemm_f8_block_plan, IN_CODES[out_fmt], rows_b, M, N, K, int(workspace_bytes))


def layernorm_bwd_workspace(M: int, N: int) -> int:
    """Workspace bytes of layernorm_bwd with dweight or dbias."""
    need = _sz(0)
    _check(_lib.layernorm_bwd_workspace(M, N, ctypes.byref(need)))
    return need.value


# ------------------------------------------------------------ allocating forms

@_on_stream
def linear_gated(A, Bg, Bu, *, bias_g=None, bias_u=None, act: str = "silu", out_dtype=None,
                 keep_preact: bool = False):
    """act(A @ Bg + bias_g) * (A @ Bu + bias_u), and with keep_preact also both factors before the
    activation (for linear_gated_backward): C or (C, gate, up).  out_dtype: A's (default) or float32."""
    _device_tensor(A, "A")
    _device_tensor(Bg, "Bg")
    out_dtype = A.dtype if out_dtype is None else out_dtype
    code, out = _formats(A, Bg, out_dtype, None)
    M, N, K = A.shape[0], Bg.shape[1], A.shape[1]
    C = _empty(M, N, out_dtype, A.device)
    G, U = (_empty(M, N, out_dtype, A.device) if keep_preact else None for _ in range(2))
    plan = _plan(_lib.gemm_gated_plan, code, out, M, N, K, _ANY)
    gemm_gated(A, Bg, Bu, C, bias_g=bias_g, bias_u=bias_u, act=act, gate=G, up=U,
               workspace=_bytes(plan["workspace_bytes"], A.device))
    return (C, G, U) if keep_preact else C


@_on_stream
def linear_gated_backward(A, Bg, Bu, dC, gate, up, *, act: str = "silu", bias: bool = False):
    """(dA, dBg, dBu, dbias_g, dbias_u) of linear_gated; the biases' are None unless `bias`."""
    _device_tensor(A, "A")
    M, N, K = _shapes(A, Bg, dC)
    code, out = _formats(A, Bg, dC.dtype, None)
    dA = _empty(M, K, A.dtype, A.device)
    dBg, dBu = (_empty(K, N, A.dtype, A.device) for _ in range(2))
    dbg, dbu = (torch.empty(N, dtype=torch.float32, device=A.device) if bias else None for _ in range(2))
    best = _sz(0)
    _check(_lib.gemm_gated_bwd_workspace(code, out, M, N, K, None, ctypes.byref(best)))
    gemm_gated_bwd(A, Bg, Bu, dC, gate, up, act=act, dA=dA, dBg=dBg, dBu=dBu, dbias_g=dbg, dbias_u=dbu,
                   workspace=_bytes(best.value, A.device))
    return dA, dBg, dBu, dbg, dbu


@_on_stream
def quantize_f8_block(X, *, rows: int = 1, transpose: bool = False):
    """(Q, scale): X, or with transpose X.T, in 8 bits with a scale per `rows` (1 or 128) x 128."""
    if rows not in (1, F8_BLOCK):
        raise ValueError("rows must be 1 or 128")
    _device_tensor(X, "X")
    M, N = X.shape
    r, c = (N, M) if transpose else (M, N)
    Q = _empty(r, c, F8, X.device)
    scale = _block_scales(r if rows == 1 else _blocks(r), c, X.device)
    quant_f8_block(X, Q, scale, transpose=transpose)
    return Q, scale


@_on_stream
def matmul_f8_block(A, B, scale_a, scale_b, *, bias=None, act: str = "none", residual=None,
                    out_dtype=torch.bfloat16):
    """act(a @ b.T + bias) + residual of float8_e4m3fn A [M, K] and B [N, K] with their blocks
    scaled, as gemm_f8_block takes them."""
    _device_tensor(A, "A")
    _device_tensor(B, "B")
    if out_dtype not in _TORCH_IN:
        raise TypeError("out_dtype must be float32, bfloat16 or float16")
    M, N, K = A.shape[0], B.shape[0], A.shape[1]
    C = _empty(M, N, out_dtype, A.device)
    plan = gemm_f8_block_plan(_TORCH_IN[out_dtype], M, N, K, _ANY, 1 if scale_b.shape[0] == N else F8_BLOCK)
    gemm_f8_block(A, B, C, scale_a, scale_b, bias=bias, act=act, residual=residual,
                  workspace=_bytes(plan["workspace_bytes"], A.device))
    return C


@_on_stream
def layer_norm(X, weight, bias=None, *, residual=None, f8=False, keep: bool = False, eps: float = 1e-5):
    """A dict of layernorm's results: "Y"; "scale" with f8 (True or "row": a scale per row;
    "block": per row and 128 columns); "total" with a residual; "mean" and "rstd" with keep
    (for layer_norm_backward)."""
    out = _norm_results(X, residual, f8)
    if keep:
        for k in ("mean", "rstd"):
            out[k] = torch.empty(X.shape[0], dtype=torch.float32, device=X.device)
    layernorm(X, weight, bias, out["Y"], residual=residual, total=out.get("total"), scale=out.get("scale"),
              mean=out.get("mean"), rstd=out.get("rstd"), eps=eps)
    return out


@_on_stream
def layer_norm_backward(dY, total, weight, mean, rstd, *, dtotal=None, bias: bool = True):
    """(dX, dweight, dbias) of layer_norm; dbias is None unless `bias`."""
    _device_tensor(dY, "dY")
    M, N = dY.shape
    dX = _empty(M, N, dY.dtype, dY.device)
    dweight = torch.empty(N, dtype=torch.float32, device=dY.device)
    dbias = torch.empty(N, dtype=torch.float32, device=dY.device) if bias else None
    layernorm_bwd(dY, total, weight, mean, rstd, dX, dtotal=dtotal, dweight=dweight, dbias=dbias,
                  workspace=_bytes(layernorm_bwd_workspace(M, N), dY.device))
    return dX, dweight, dbias
