"""Binding of the linear layer's operators (include/dgemm.h): products
with bias, activation and residual and their gradients, 8-bit products, norms
and quantizers.  As in _binding, the functions named like the C entry points
(in _marshal, csrc/marshal.cpp) only marshal tensors the caller has allocated;
the host queries go through ctypes; `linear`, `linear_backward`,
`matmul_f8`, `rms_norm`, `rms_norm_backward` and `quantize_f8` allocate their
results and workspaces the way `matmul` does.

Nothing is recorded for autograd (nor by `matmul`): results never require
gradients, whatever the inputs do, and a training program calls
`linear_backward` and `rms_norm_backward` itself."""
import ctypes
import functools
import inspect

import torch

from ._binding import DGEMM_OUT_F32, DGEMM_OUT_SAME, IN_CODES, _TORCH_IN, _check, _lib, _shapes
from ._marshal import (  # noqa: F401
    gemm_act, gemm_act_bwd, gemm_f8, quant_f8, rmsnorm, rmsnorm_bwd,
)

_i, _p, _sz, _f = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
_P, _PS = ctypes.POINTER(_i), ctypes.POINTER(_sz)
_ARGTYPES = {
    "gemm_act": [_i] * 5 + [_p, _i] * 3 + [_p, _i, _p, _i, _p, _i, _p, _sz, _p],
    "gemm_act_plan": [_i] * 5 + [_sz, _P, _P, _P, _PS],
    "gemm_act_bwd": [_i] * 5 + [_p, _i] * 4 + [_i] + [_p, _i] * 2 + [_p, _p, _sz, _p],
    "gemm_act_bwd_workspace": [_i] * 6 + [_PS, _PS],
    "gemm_f8": [_i] * 4 + [_p, _i] * 3 + [_p, _p, _p, _i, _p, _i, _p, _sz, _p],
    "gemm_f8_plan": [_i] * 4 + [_sz, _P, _P, _P, _PS],
    "rmsnorm": [_i] * 4 + [_p, _i] * 3 + [_p, _f, _p, _i, _p, _p, _p],
    "rmsnorm_bwd": [_i] * 3 + [_p, _i] * 2 + [_p, _p] + [_p, _i] * 2 + [_p, _p, _sz, _p],
    "rmsnorm_bwd_workspace": [_i, _i, _PS],
    "quant_f8": [_i] * 4 + [_p, _i] * 2 + [_p, _p],
}
for _name, _types in _ARGTYPES.items():
    getattr(_lib, _name).argtypes = _types
    getattr(_lib, _name).restype = _i

ACT_CODES = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
F8 = torch.float8_e4m3fn
_ANY = 1 << 40  # a workspace size that no plan exceeds


def _act(act: str) -> int:
    if act not in ACT_CODES:
        raise ValueError(f"act must be one of {', '.join(ACT_CODES)}")
    return ACT_CODES[act]


def _formats(A, B, C_dtype, in_fmt):
    """(input code, output code) of a product of A and B with C_dtype results."""
    dtype = A.dtype
    own = _TORCH_IN.get(dtype)
    fmt = in_fmt or own
    if own is None or B.dtype is not dtype or (fmt != own and not (fmt == "f32x3" and own == "f32")):
        raise TypeError("unsupported input dtypes")
    if C_dtype is torch.float32:
        return IN_CODES[fmt], DGEMM_OUT_F32
    if C_dtype is not dtype:
        raise TypeError("C must be float32 or the input dtype")
    return IN_CODES[fmt], DGEMM_OUT_SAME


def _device_tensor(t, name):
    if t.dim() != 2:
        raise ValueError("operands must be 2-D")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")


def _plan(fn, *args) -> dict:
    v = [ctypes.c_int(-1) for _ in range(3)]
    used = _sz(0)
    _check(fn(*args, *[ctypes.byref(x) for x in v], ctypes.byref(used)))
    return {"tile_rows": v[0].value, "tile_cols": v[1].value, "splits": v[2].value,
            "workspace_bytes": used.value}


def gemm_act_plan(in_fmt: str, M: int, N: int, K: int, workspace_bytes: int,
                  out_same: bool = False) -> dict:
    """Host query of the plan gemm_act uses with `workspace_bytes` available."""
    return _plan(_lib.gemm_act_plan, IN_CODES[in_fmt], DGEMM_OUT_SAME if out_same else DGEMM_OUT_F32,
                 M, N, K, int(workspace_bytes))


def gemm_f8_plan(out_fmt: str, M: int, N: int, K: int, workspace_bytes: int) -> dict:
    """Host query of the plan gemm_f8 uses with `workspace_bytes` available."""
    return _plan(_lib.gemm_f8_plan, IN_CODES[out_fmt], M, N, K, int(workspace_bytes))


def gemm_act_bwd_workspace(in_fmt: str, M: int, N: int, K: int, act: str = "none",
                           out_same: bool = True):
    """(required, best) workspace bytes of gemm_act_bwd."""
    req, best = _sz(0), _sz(0)
    _check(_lib.gemm_act_bwd_workspace(IN_CODES[in_fmt], DGEMM_OUT_SAME if out_same else DGEMM_OUT_F32,
                                       M, N, K, _act(act), ctypes.byref(req), ctypes.byref(best)))
    return req.value, best.value


def rmsnorm_bwd_workspace(M: int, N: int) -> int:
    """Workspace bytes of rmsnorm_bwd with dweight."""
    need = _sz(0)
    _check(_lib.rmsnorm_bwd_workspace(M, N, ctypes.byref(need)))
    return need.value


# ------------------------------------------------------------ allocating forms

def _empty(rows: int, cols: int, dtype, device) -> torch.Tensor:
    """A matrix whose row pitch is a multiple of 16 bytes."""
    per16 = 16 // torch.empty((), dtype=dtype).element_size()
    return torch.empty((rows, (cols + per16 - 1) // per16 * per16), dtype=dtype, device=device)[:, :cols]


def _bytes(n: int, device):
    return torch.empty(n, dtype=torch.uint8, device=device) if n > 0 else None


def _on_stream(fn):
    """Adds `stream=None`: runs fn with it current, so that its results and workspaces
    come from the allocator's pool of the stream the kernels run on (as matmul does)."""
    sig = inspect.signature(fn)
    first = next(iter(sig.parameters))

    @functools.wraps(fn)
    def wrapped(*args, stream=None, **kw):
        if stream is not None and (args or first in kw):
            device = (args[0] if args else kw[first]).device
            if stream != torch.cuda.current_stream(device):
                with torch.cuda.stream(stream):
                    return fn(*args, **kw)
        return fn(*args, **kw)
    wrapped.__signature__ = sig.replace(parameters=[
        *sig.parameters.values(), inspect.Parameter("stream", inspect.Parameter.KEYWORD_ONLY, default=None)])
    return wrapped


@_on_stream
def linear(A, B, *, bias=None, act: str = "none", residual=None, out_dtype=None,
           keep_preact: bool = False, in_fmt: str = None):
    """act(A @ B + bias) + residual, and with keep_preact also A @ B + bias (for
    linear_backward): C or (C, Z).  out_dtype: A's (default) or float32."""
    _device_tensor(A, "A")
    _device_tensor(B, "B")
    out_dtype = A.dtype if out_dtype is None else out_dtype
    code, out = _formats(A, B, out_dtype, in_fmt)
    M, N, K = A.shape[0], B.shape[1], A.shape[1]
    C = _empty(M, N, out_dtype, A.device)
    Z = _empty(M, N, out_dtype, A.device) if keep_preact else None
    plan = _plan(_lib.gemm_act_plan, code, out, M, N, K, _ANY)
    gemm_act(A, B, C, bias=bias, act=act, residual=residual, preact=Z,
             workspace=_bytes(plan["workspace_bytes"], A.device), in_fmt=in_fmt)
    return (C, Z) if keep_preact else C


@_on_stream
def linear_backward(A, B, dC, *, preact=None, act: str = "none", bias: bool = False,
                    in_fmt: str = None):
    """(dA, dB, dbias) of linear; dbias is None unless `bias`.  The residual's
    gradient is dC itself."""
    M, N, K = _shapes(A, B, dC)
    code, out = _formats(A, B, dC.dtype, in_fmt)
    dA, dB = _empty(M, K, A.dtype, A.device), _empty(K, N, A.dtype, A.device)
    dbias = torch.empty(N, dtype=torch.float32, device=A.device) if bias else None
    best = _sz(0)
    _check(_lib.gemm_act_bwd_workspace(code, out, M, N, K, _act(act), None, ctypes.byref(best)))
    gemm_act_bwd(A, B, dC, dA=dA, dB=dB, dbias=dbias, preact=preact, act=act,
                 workspace=_bytes(best.value, A.device), in_fmt=in_fmt)
    return dA, dB, dbias


@_on_stream
def matmul_f8(A, B, scale_a, scale_b, *, bias=None, act: str = "none", residual=None,
              out_dtype=torch.bfloat16):
    """act(scale_a[:, None] * scale_b * (A @ B.T) + bias) + residual of
    float8_e4m3fn A [M, K] and B [N, K]."""
    _device_tensor(A, "A")
    _device_tensor(B, "B")
    if out_dtype not in _TORCH_IN:
        raise TypeError("out_dtype must be float32, bfloat16 or float16")
    M, N, K = A.shape[0], B.shape[0], A.shape[1]
    C = _empty(M, N, out_dtype, A.device)
    plan = gemm_f8_plan(_TORCH_IN[out_dtype], M, N, K, _ANY)
    gemm_f8(A, B, C, scale_a, scale_b, bias=bias, act=act, residual=residual,
            workspace=_bytes(plan["workspace_bytes"], A.device))
    return C


@_on_stream
def rms_norm(X, weight, *, residual=None, f8: bool = False, keep: bool = False, eps: float = 1e-6):
    """A dict of rmsnorm's results: "Y"; "scale" with f8; "total" with a residual;
    "rstd" with keep (for rms_norm_backward)."""
    _device_tensor(X, "X")
    M, N = X.shape
    out = {"Y": _empty(M, N, F8 if f8 else X.dtype, X.device)}
    if f8:
        out["scale"] = torch.empty(M, dtype=torch.float32, device=X.device)
    if residual is not None:
        out["total"] = _empty(M, N, X.dtype, X.device)
    if keep:
        out["rstd"] = torch.empty(M, dtype=torch.float32, device=X.device)
    rmsnorm(X, weight, out["Y"], residual=residual, total=out.get("total"), scale=out.get("scale"),
            rstd=out.get("rstd"), eps=eps)
    return out


@_on_stream
def rms_norm_backward(dY, total, weight, rstd, *, dtotal=None):
    """(dX, dweight) of rms_norm."""
    _device_tensor(dY, "dY")
    M, N = dY.shape
    dX = _empty(M, N, dY.dtype, dY.device)
    dweight = torch.empty(N, dtype=torch.float32, device=dY.device)
    rmsnorm_bwd(dY, total, weight, rstd, dX, dtotal=dtotal, dweight=dweight,
                workspace=_bytes(rmsnorm_bwd_workspace(M, N), dY.device))
    return dX, dweight


@_on_stream
def quantize_f8(X, *, transpose: bool = False):
    """(Q, scale): X's rows (with transpose its columns, transposed) in 8 bits."""
    _device_tensor(X, "X")
    M, N = X.shape
    rows, cols = (N, M) if transpose else (M, N)
    Q = _empty(rows, cols, F8, X.device)
    scale = torch.empty(rows, dtype=torch.float32, device=X.device)
    quant_f8(X, Q, scale, transpose=transpose)
    return Q, scale
