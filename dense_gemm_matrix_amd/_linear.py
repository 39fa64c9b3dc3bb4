"""ctypes binding of the linear layer's operators (include/dgemm.h): products
with bias, activation and residual and their gradients, 8-bit products, norms
and quantizers.  As in _binding, the functions named like the C entry points
only marshal tensors the caller has allocated; `linear`, `linear_backward`,
`matmul_f8`, `rms_norm`, `rms_norm_backward` and `quantize_f8` allocate their
results and workspaces the way `matmul` does."""
import ctypes

import torch

from ._binding import (DGEMM_OUT_F32, DGEMM_OUT_SAME, IN_CODES, _TORCH_IN, _check, _lib, _on_device,
                       _pitch, _shapes, _stream)

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


def _vector(t, n: int, device, name: str):
    """Pointer of an optional fp32 vector of length n."""
    if t is None:
        return None
    if t.dtype != torch.float32 or t.dim() != 1 or t.numel() != n or not t.is_contiguous() \
            or t.device != device:
        raise ValueError(f"{name} must be a contiguous float32 device vector of length {n}")
    return t.data_ptr()


def _matrix(t, shape, dtype, device, name: str):
    """(pointer, pitch) of an optional matrix operand."""
    if t is None:
        return None, 0
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if tuple(t.shape) != tuple(shape) or t.device != device:
        raise ValueError(f"{name} must be a {tuple(shape)} matrix on {device}")
    return t.data_ptr(), _pitch(t, shape[1])


def _workspace(ws, device):
    if ws is None:
        return None, 0
    if ws.device != device or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the output's device")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _formats(A, B, C_dtype, in_fmt):
    """(input code, output code) of a product of A and B with C_dtype results."""
    fmt = in_fmt or _TORCH_IN.get(A.dtype)
    if fmt not in IN_CODES or B.dtype != A.dtype or _TORCH_IN.get(A.dtype) != ("f32" if fmt == "f32x3" else fmt):
        raise TypeError("unsupported input dtypes")
    if C_dtype == torch.float32:
        return IN_CODES[fmt], DGEMM_OUT_F32
    if C_dtype != A.dtype:
        raise TypeError("C must be float32 or the input dtype")
    return IN_CODES[fmt], DGEMM_OUT_SAME


def _device_tensor(t, name):
    if t.dim() != 2:
        raise ValueError("operands must be 2-D")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")


def gemm_act(A: torch.Tensor, B: torch.Tensor, C: torch.Tensor, *, bias: torch.Tensor = None,
             act: str = "none", residual: torch.Tensor = None, preact: torch.Tensor = None,
             workspace: torch.Tensor = None, in_fmt: str = None, stream=None) -> None:
    """C = act(A @ B + bias) + residual; preact (optional) = A @ B + bias.

    `residual` and `preact` have C's shape and dtype; `residual` may be C itself.
    `workspace` and `in_fmt` as in gemm_ex."""
    M, N, K = _shapes(A, B, C)
    code, out = _formats(A, B, C.dtype, in_fmt)
    r, ldr = _matrix(residual, (M, N), C.dtype, C.device, "residual")
    z, ldz = _matrix(preact, (M, N), C.dtype, C.device, "preact")
    ws, ws_bytes = _workspace(workspace, C.device)
    with _on_device(C):
        _check(_lib.gemm_act(code, out, M, N, K, A.data_ptr(), _pitch(A, K), B.data_ptr(),
                             _pitch(B, N), C.data_ptr(), _pitch(C, N),
                             _vector(bias, N, C.device, "bias"), _act(act), r, ldr, z, ldz, ws,
                             ws_bytes, _stream(C, stream)))


def gemm_act_bwd(A: torch.Tensor, B: torch.Tensor, dC: torch.Tensor, *, dA: torch.Tensor = None,
                 dB: torch.Tensor = None, dbias: torch.Tensor = None, preact: torch.Tensor = None,
                 act: str = "none", workspace: torch.Tensor = None, in_fmt: str = None,
                 stream=None) -> None:
    """Gradients of gemm_act: dA (A's shape and dtype), dB (B's) and dbias
    (float32), each written if given; `preact` as gemm_act stored it (not needed
    with act "none").  The workspace is at least gemm_act_bwd_workspace's."""
    M, N, K = _shapes(A, B, dC)
    code, out = _formats(A, B, dC.dtype, in_fmt)
    a = _act(act)
    if a and preact is None:
        raise ValueError("the gradient of an activation needs preact")
    z, ldz = _matrix(preact if a else None, (M, N), dC.dtype, dC.device, "preact")
    da, ldda = _matrix(dA, (M, K), A.dtype, dC.device, "dA")
    db, lddb = _matrix(dB, (K, N), A.dtype, dC.device, "dB")
    ws, ws_bytes = _workspace(workspace, dC.device)
    with _on_device(dC):
        _check(_lib.gemm_act_bwd(code, out, M, N, K, A.data_ptr(), _pitch(A, K), B.data_ptr(),
                                 _pitch(B, N), dC.data_ptr(), _pitch(dC, N), z, ldz, a, da, ldda,
                                 db, lddb, _vector(dbias, N, dC.device, "dbias"), ws, ws_bytes,
                                 _stream(dC, stream)))


def gemm_f8(A: torch.Tensor, B: torch.Tensor, C: torch.Tensor, scale_a: torch.Tensor,
            scale_b: torch.Tensor, *, bias: torch.Tensor = None, act: str = "none",
            residual: torch.Tensor = None, workspace: torch.Tensor = None, stream=None) -> None:
    """C = act(scale_a[:, None] * scale_b * (A @ B.T) + bias) + residual for
    float8_e4m3fn A [M, K] and B [N, K]; C (and residual) fp32, bf16 or fp16."""
    for name, t in (("A", A), ("B", B), ("C", C)):
        _device_tensor(t, name)
    M, K = A.shape
    N = B.shape[0]
    if B.shape[1] != K or tuple(C.shape) != (M, N):
        raise ValueError(f"shapes {tuple(A.shape)} x {tuple(B.shape)}^T -> {tuple(C.shape)}")
    if not (A.device == B.device == C.device):
        raise ValueError(f"operands on different devices: {A.device}, {B.device}, {C.device}")
    if A.dtype != F8 or B.dtype != F8:
        raise TypeError(f"A and B must be {F8}")
    if C.dtype not in _TORCH_IN:
        raise TypeError("C must be float32, bfloat16 or float16")
    if scale_a is None or scale_b is None:
        raise ValueError("scale_a and scale_b are required")
    r, ldr = _matrix(residual, (M, N), C.dtype, C.device, "residual")
    ws, ws_bytes = _workspace(workspace, C.device)
    with _on_device(C):
        _check(_lib.gemm_f8(IN_CODES[_TORCH_IN[C.dtype]], M, N, K, A.data_ptr(), _pitch(A, K),
                            B.data_ptr(), _pitch(B, K), C.data_ptr(), _pitch(C, N),
                            _vector(scale_a, M, C.device, "scale_a"),
                            _vector(scale_b, N, C.device, "scale_b"),
                            _vector(bias, N, C.device, "bias"), _act(act), r, ldr, ws, ws_bytes,
                            _stream(C, stream)))


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


def rmsnorm(X: torch.Tensor, weight: torch.Tensor, Y: torch.Tensor, *, residual: torch.Tensor = None,
            total: torch.Tensor = None, scale: torch.Tensor = None, rstd: torch.Tensor = None,
            eps: float = 1e-6, stream=None) -> None:
    """Y = s * rstd * weight row by row, s = X + residual, rstd = (mean s^2 + eps)^-1/2.

    Y has X's dtype, or is float8_e4m3fn with a float32 `scale` per row (gemm_f8's
    A and scale_a).  `total` (X's dtype) receives s and `rstd` (float32, one per
    row) its root where given: what rmsnorm_bwd reads.  `total` and Y may be X or
    residual themselves."""
    _device_tensor(X, "X")
    M, N = X.shape
    if X.dtype not in _TORCH_IN:
        raise TypeError("X must be float32, bfloat16 or float16")
    f8 = Y.dtype == F8
    if f8 != (scale is not None):
        raise ValueError("a float8_e4m3fn Y takes a scale, and only that")
    if weight is None:
        raise ValueError("weight is required")
    y, ldy = _matrix(Y, (M, N), F8 if f8 else X.dtype, X.device, "Y")
    r, ldr = _matrix(residual, (M, N), X.dtype, X.device, "residual")
    s, lds = _matrix(total, (M, N), X.dtype, X.device, "total")
    with _on_device(X):
        _check(_lib.rmsnorm(IN_CODES[_TORCH_IN[X.dtype]], int(f8), M, N, X.data_ptr(), _pitch(X, N), r,
                            ldr, s, lds, _vector(weight, N, X.device, "weight"), float(eps), y, ldy,
                            _vector(scale, M, X.device, "scale"), _vector(rstd, M, X.device, "rstd"),
                            _stream(X, stream)))


def rmsnorm_bwd(dY: torch.Tensor, total: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                dX: torch.Tensor, *, dtotal: torch.Tensor = None, dweight: torch.Tensor = None,
                workspace: torch.Tensor = None, stream=None) -> None:
    """Gradients of rmsnorm: dX (the residual's too) and, where given, dweight
    (float32; needs rmsnorm_bwd_workspace's bytes).  `total` and `rstd` as rmsnorm
    stored them (total is X where there was no residual); `dtotal` is the
    gradient that reaches total by other ways.  dX may be dY or dtotal itself."""
    _device_tensor(dY, "dY")
    M, N = dY.shape
    if dY.dtype not in _TORCH_IN:
        raise TypeError("dY must be float32, bfloat16 or float16")
    if weight is None or rstd is None:
        raise ValueError("weight and rstd are required")
    s, lds = _matrix(total, (M, N), dY.dtype, dY.device, "total")
    d, ldd = _matrix(dtotal, (M, N), dY.dtype, dY.device, "dtotal")
    x, ldx = _matrix(dX, (M, N), dY.dtype, dY.device, "dX")
    ws, ws_bytes = _workspace(workspace, dY.device)
    with _on_device(dY):
        _check(_lib.rmsnorm_bwd(IN_CODES[_TORCH_IN[dY.dtype]], M, N, dY.data_ptr(), _pitch(dY, N), s,
                                lds, _vector(weight, N, dY.device, "weight"),
                                _vector(rstd, M, dY.device, "rstd"), d, ldd, x, ldx,
                                _vector(dweight, N, dY.device, "dweight"), ws, ws_bytes,
                                _stream(dY, stream)))


def rmsnorm_bwd_workspace(M: int, N: int) -> int:
    """Workspace bytes of rmsnorm_bwd with dweight."""
    need = _sz(0)
    _check(_lib.rmsnorm_bwd_workspace(M, N, ctypes.byref(need)))
    return need.value


def quant_f8(X: torch.Tensor, Q: torch.Tensor, scale: torch.Tensor, *, transpose: bool = False,
             stream=None) -> None:
    """Q, scale = X's rows in 8 bits (float8_e4m3fn, one float32 scale per row);
    with transpose its columns, Q being X.T's shape: gemm_f8's B from a [K, N]
    weight."""
    _device_tensor(X, "X")
    M, N = X.shape
    if X.dtype not in _TORCH_IN:
        raise TypeError("X must be float32, bfloat16 or float16")
    if scale is None:
        raise ValueError("scale is required")
    q, ldq = _matrix(Q, (N, M) if transpose else (M, N), F8, X.device, "Q")
    with _on_device(X):
        _check(_lib.quant_f8(IN_CODES[_TORCH_IN[X.dtype]], int(transpose), M, N, X.data_ptr(),
                             _pitch(X, N), q, ldq,
                             _vector(scale, N if transpose else M, X.device, "scale"),
                             _stream(X, stream)))


# ------------------------------------------------------------ allocating forms

def _empty(rows: int, cols: int, dtype, device) -> torch.Tensor:
    """A matrix whose row pitch is a multiple of 16 bytes."""
    per16 = 16 // torch.empty((), dtype=dtype).element_size()
    return torch.empty((rows, (cols + per16 - 1) // per16 * per16), dtype=dtype, device=device)[:, :cols]


def _bytes(n: int, device):
    return torch.empty(n, dtype=torch.uint8, device=device) if n > 0 else None


def _on_stream(fn):
    """Runs fn with `stream` current, so that its results and workspaces come from
    the allocator's pool of the stream the kernels run on (as matmul does)."""
    def wrapped(X, *args, stream=None, **kw):
        if stream is not None and stream != torch.cuda.current_stream(X.device):
            with torch.cuda.stream(stream):
                return fn(X, *args, **kw)
        return fn(X, *args, **kw)
    wrapped.__name__, wrapped.__doc__ = fn.__name__, fn.__doc__
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
