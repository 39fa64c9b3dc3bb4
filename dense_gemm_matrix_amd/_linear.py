"""ctypes binding of the linear layer's operators (include/dgemm.h): products
with bias, activation and residual and their gradients, 8-bit products, norms
and quantizers.  As in _binding, the functions named like the C entry points
only marshal tensors the caller has allocated; `linear`, `linear_backward`,
`matmul_f8`, `rms_norm`, `rms_norm_backward` and `quantize_f8` allocate their
results and workspaces the way `matmul` does."""
import ctypes

import torch

from ._binding import (DGEMM_OUT_F32, DGEMM_OUT_SAME, IN_CODES, _TORCH_IN, _check, _lib, _on_device,
                       _shapes, _stream)

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


# The checks below run on every call and are most of a small call's host time, so
# each is one pass over attributes that torch answers without building objects
# (device indices, dtypes and sizes compared as such), and the messages are made
# only when one fails.
_FP32 = torch.float32
_PER16 = {torch.float32: 4, torch.bfloat16: 8, torch.float16: 8, F8: 16}
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") \
    else torch.cuda.current_device


def _vector(t, n: int, dev: int, name: str):
    """Pointer of an optional fp32 vector of length n on device index dev."""
    if t is None:
        return None
    if t.dtype is not _FP32 or t.dim() != 1 or t.numel() != n or not t.is_contiguous() \
            or t.get_device() != dev:
        raise ValueError(f"{name} must be a contiguous float32 device vector of length {n}")
    return t.data_ptr()


def _ld(t, rows: int, cols: int) -> int:
    """_pitch, for a matrix of known size."""
    pitch, inner = t.stride()
    if inner != 1 and cols > 1 and rows > 0:
        raise ValueError("operands must be row-major with unit inner stride")
    if rows > 1:
        return pitch
    per16 = _PER16[t.dtype]
    return (max(cols, 1) + per16 - 1) // per16 * per16


def _matrix(t, rows: int, cols: int, dtype, dev: int, name: str):
    """(pointer, pitch) of an optional matrix operand on device index dev."""
    if t is None:
        return None, 0
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape != (rows, cols) or t.get_device() != dev:
        raise ValueError(f"{name} must be a {(rows, cols)} matrix on device {dev}")
    return t.data_ptr(), _ld(t, rows, cols)


def _workspace(ws, dev: int):
    if ws is None:
        return None, 0
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the output's device")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _call(fn, t, *args) -> None:
    """Calls a C entry point with t's device current."""
    if t.get_device() == _current_device():
        status = fn(*args)
    else:
        with _on_device(t):
            status = fn(*args)
    if status:
        _check(status)


def _formats(A, B, C_dtype, in_fmt):
    """(input code, output code) of a product of A and B with C_dtype results."""
    dtype = A.dtype
    own = _TORCH_IN.get(dtype)
    fmt = in_fmt or own
    if own is None or B.dtype is not dtype or (fmt != own and not (fmt == "f32x3" and own == "f32")):
        raise TypeError("unsupported input dtypes")
    if C_dtype is _FP32:
        return IN_CODES[fmt], DGEMM_OUT_F32
    if C_dtype is not dtype:
        raise TypeError("C must be float32 or the input dtype")
    return IN_CODES[fmt], DGEMM_OUT_SAME


def _device_tensor(t, name):
    if t.dim() != 2:
        raise ValueError("operands must be 2-D")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")


def _sizes(A, B, C):
    """_shapes, for the calls of this module."""
    sa, sb = A.shape, B.shape
    if len(sa) != 2 or len(sb) != 2 or sa[1] != sb[0] or C.shape != (sa[0], sb[1]) \
            or not (A.get_device() == B.get_device() == C.get_device() >= 0):
        return _shapes(A, B, C)  # raises
    return sa[0], sb[1], sa[1]


def gemm_act(A: torch.Tensor, B: torch.Tensor, C: torch.Tensor, *, bias: torch.Tensor = None,
             act: str = "none", residual: torch.Tensor = None, preact: torch.Tensor = None,
             workspace: torch.Tensor = None, in_fmt: str = None, stream=None) -> None:
    """C = act(A @ B + bias) + residual; preact (optional) = A @ B + bias.

    `residual` and `preact` have C's shape and dtype; `residual` may be C itself.
    `workspace` and `in_fmt` as in gemm_ex."""
    M, N, K = _sizes(A, B, C)
    code, out = _formats(A, B, C.dtype, in_fmt)
    dev, dtype = C.get_device(), C.dtype
    r, ldr = _matrix(residual, M, N, dtype, dev, "residual")
    z, ldz = _matrix(preact, M, N, dtype, dev, "preact")
    ws, ws_bytes = _workspace(workspace, dev)
    _call(_lib.gemm_act, C, code, out, M, N, K, A.data_ptr(), _ld(A, M, K), B.data_ptr(),
          _ld(B, K, N), C.data_ptr(), _ld(C, M, N), _vector(bias, N, dev, "bias"), _act(act), r, ldr, z,
          ldz, ws, ws_bytes, _stream(C, stream))


def gemm_act_bwd(A: torch.Tensor, B: torch.Tensor, dC: torch.Tensor, *, dA: torch.Tensor = None,
                 dB: torch.Tensor = None, dbias: torch.Tensor = None, preact: torch.Tensor = None,
                 act: str = "none", workspace: torch.Tensor = None, in_fmt: str = None,
                 stream=None) -> None:
    """Gradients of gemm_act: dA (A's shape and dtype), dB (B's) and dbias
    (float32), each written if given; `preact` as gemm_act stored it (not needed
    with act "none").  The workspace is at least gemm_act_bwd_workspace's."""
    M, N, K = _sizes(A, B, dC)
    code, out = _formats(A, B, dC.dtype, in_fmt)
    a = _act(act)
    if a and preact is None:
        raise ValueError("the gradient of an activation needs preact")
    dev = dC.get_device()
    z, ldz = _matrix(preact if a else None, M, N, dC.dtype, dev, "preact")
    da, ldda = _matrix(dA, M, K, A.dtype, dev, "dA")
    db, lddb = _matrix(dB, K, N, A.dtype, dev, "dB")
    ws, ws_bytes = _workspace(workspace, dev)
    _call(_lib.gemm_act_bwd, dC, code, out, M, N, K, A.data_ptr(), _ld(A, M, K), B.data_ptr(),
          _ld(B, K, N), dC.data_ptr(), _ld(dC, M, N), z, ldz, a, da, ldda, db, lddb,
          _vector(dbias, N, dev, "dbias"), ws, ws_bytes, _stream(dC, stream))


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
    dev = C.get_device()
    if not (A.get_device() == B.get_device() == dev):
        raise ValueError(f"operands on different devices: {A.device}, {B.device}, {C.device}")
    if A.dtype is not F8 or B.dtype is not F8:
        raise TypeError(f"A and B must be {F8}")
    if C.dtype not in _TORCH_IN:
        raise TypeError("C must be float32, bfloat16 or float16")
    if scale_a is None or scale_b is None:
        raise ValueError("scale_a and scale_b are required")
    r, ldr = _matrix(residual, M, N, C.dtype, dev, "residual")
    ws, ws_bytes = _workspace(workspace, dev)
    _call(_lib.gemm_f8, C, IN_CODES[_TORCH_IN[C.dtype]], M, N, K, A.data_ptr(), _ld(A, M, K),
          B.data_ptr(), _ld(B, N, K), C.data_ptr(), _ld(C, M, N), _vector(scale_a, M, dev, "scale_a"),
          _vector(scale_b, N, dev, "scale_b"), _vector(bias, N, dev, "bias"), _act(act), r, ldr, ws,
          ws_bytes, _stream(C, stream))


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
    f8 = Y.dtype is F8
    if f8 != (scale is not None):
        raise ValueError("a float8_e4m3fn Y takes a scale, and only that")
    if weight is None:
        raise ValueError("weight is required")
    dev, dtype = X.get_device(), X.dtype
    y, ldy = _matrix(Y, M, N, F8 if f8 else dtype, dev, "Y")
    r, ldr = _matrix(residual, M, N, dtype, dev, "residual")
    s, lds = _matrix(total, M, N, dtype, dev, "total")
    _call(_lib.rmsnorm, X, IN_CODES[_TORCH_IN[dtype]], int(f8), M, N, X.data_ptr(), _ld(X, M, N), r, ldr,
          s, lds, _vector(weight, N, dev, "weight"), eps, y, ldy, _vector(scale, M, dev, "scale"),
          _vector(rstd, M, dev, "rstd"), _stream(X, stream))


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
    dev, dtype = dY.get_device(), dY.dtype
    s, lds = _matrix(total, M, N, dtype, dev, "total")
    d, ldd = _matrix(dtotal, M, N, dtype, dev, "dtotal")
    x, ldx = _matrix(dX, M, N, dtype, dev, "dX")
    ws, ws_bytes = _workspace(workspace, dev)
    _call(_lib.rmsnorm_bwd, dY, IN_CODES[_TORCH_IN[dtype]], M, N, dY.data_ptr(), _ld(dY, M, N), s, lds,
          _vector(weight, N, dev, "weight"), _vector(rstd, M, dev, "rstd"), d, ldd, x, ldx,
          _vector(dweight, N, dev, "dweight"), ws, ws_bytes, _stream(dY, stream))


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
    dev = X.get_device()
    qrows, qcols = (N, M) if transpose else (M, N)
    q, ldq = _matrix(Q, qrows, qcols, F8, dev, "Q")
    _call(_lib.quant_f8, X, IN_CODES[_TORCH_IN[X.dtype]], int(transpose), M, N, X.data_ptr(),
          _ld(X, M, N), q, ldq, _vector(scale, qrows, dev, "scale"), _stream(X, stream))


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
    M, N, K = _sizes(A, B, dC)
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
