"""Plain 64-bit forms of the linear layer's operators for the tests, and the
error bounds the kernels are held to."""
import math

import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half steps
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}
SLOPE = 1.13   # the largest |act'|: GELU's 1.129
F8 = torch.float8_e4m3fn


def act64(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return 0.5 * z * torch.erfc(-z / math.sqrt(2.0))
    if act == "gelu_tanh":
        return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def act_grad64(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * torch.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        s = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        return s + z * s * (1.0 - s) * c * (1.0 + 3.0 * 0.044715 * z * z)
    if act == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1.0 - s)
    return torch.ones_like(z)


def sum_bound(K, S, x3=False):
    """fp32 summation of K products in any order: at most K half steps of the
    absolute sum S, and two more for the scales or the product's rounding; the
    3 x bf16 path drops at most 3 * 2^-16 of each product."""
    return (K + 2) * 2.0 ** -24 * S + (3.0 * 2.0 ** -16 * S if x3 else 0.0)


def linear64(A, B, bias, act, R):
    """(C, Z, S): S the sum of absolute products and of the bias."""
    A, B = A.double(), B.double()
    Z, S = A @ B, A.abs() @ B.abs()
    if bias is not None:
        Z = Z + bias.double()
        S = S + bias.double().abs()
    C = act64(Z, act)
    return (C if R is None else C + R.double()), Z, S


def out_bound(C, Z, dz, R, dtype, act):
    """Bound of an output act(z) + r whose fp32 z is off by at most dz: the
    activation passes on SLOPE dz and is itself evaluated in fp32, within 32
    half steps of |z| (its exponent's argument, up to a few times |z|, and some
    six operations on values of at most |z|); one rounding of the residual's sum
    and one to the output's format."""
    e = dz if act == "none" else SLOPE * dz + 32 * 2.0 ** -24 * Z.abs()
    if R is not None:
        e = e + 2.0 ** -24 * C.abs() + 2.0 ** -24 * act64(Z, act).abs()
    return e + U[dtype] * (C.abs() + e) + TINY[dtype]


def within(x, ref, bound):
    x = x.detach().cpu().double()
    bad = ~((x - ref).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst " \
        f"{float(((x - ref).abs() / bound).nan_to_num(9e99).max()):.3g} x the bound"


def quant64(y):
    """Rows in 8 bits as doubles: (Q, scale)."""
    scale = (y.abs().amax(dim=1) / 448.0).clamp_min(2.0 ** -100)
    v = y / scale[:, None]
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(1e-300))).clamp_min(-6.0) - 3.0)
    return torch.round(v / step) * step, scale


def padded(x, dtype, extra=0, fill=float("nan"), device="cuda"):
    """x as a view of a buffer with row pitches of 16-byte multiples (`extra` more
    16-byte pieces), the gap holding `fill`."""
    rows, cols = x.shape
    per16 = 16 // torch.empty((), dtype=dtype).element_size()
    pitch = ((cols + per16 - 1) // per16 + extra) * per16
    buf = torch.full((rows, pitch), fill, dtype=torch.float32).to(dtype)
    buf[:, :cols] = x.to(dtype)
    return buf.to(device)[:, :cols]


def sentinel(rows, cols, dtype, extra=1, device="cuda"):
    """An output buffer full of NaN, and its gap."""
    return padded(torch.full((rows, cols), float("nan")), dtype, extra, device=device)


def gap_kept(t):
    rows, cols = t.shape
    if rows == 0:
        return True
    full = torch.as_strided(t, (rows, t.stride(0)), (t.stride(0), 1), t.storage_offset())
    return bool(torch.isnan(full[:-1, cols:].float()).all()) if rows > 1 else True
