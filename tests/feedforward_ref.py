"""Plain 64-bit forms of the feed-forward block's operators for the tests, and the
error bounds the kernels are held to."""
import torch

from tests.linear_ref import F8, TINY, U

H = 2.0 ** -24  # an fp32 half step, relative


def blocks(n):
    return (n + 127) // 128


def quant_block64(x, rows):
    """(codes as doubles, fp32 scales) of x with a scale per rows x 128: scales are fp32 quotients, codes the
    nearest e4m3 values of the exact quotients by them."""
    r, c = x.shape
    rb, cb = -(-r // rows), blocks(c)
    p = torch.zeros(rb * rows, cb * 128, dtype=torch.float64)
    p[:r, :c] = x.double()
    p = p.view(rb, rows, cb, 128)
    scale = (p.abs().amax((1, 3)).float() / torch.tensor(448.0)).clamp_min(2.0 ** -100)
    v = p / scale.double()[:, None, :, None]
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(1e-300))).clamp_min(-6.0) - 3.0)
    q = (torch.round(v / step) * step).clamp(-448.0, 448.0).reshape(rb * rows, cb * 128)[:r, :c]
    return q, scale


def spread(scale, rows, r, c):
    """Block scales to every element."""
    return scale.double().repeat_interleave(rows, 0)[:r].repeat_interleave(128, 1)[:, :c]


def block_product64(A, B, sa, sb, rows_b):
    """(product, sum of absolute products, what the 8-bit instruction may drop) of e4m3 A and B with block scales:
    of each product, what lies below 2^-13 of the largest of the block."""
    M, K, N = A.shape[0], A.shape[1], B.shape[0]
    a, b = A.double() * spread(sa, 1, M, K), B.double() * spread(sb, rows_b, N, K)
    drop = torch.zeros(M, N, dtype=torch.float64)
    for k in range(0, K, 128):
        x, y = a[:, k:k + 128].abs(), b[:, k:k + 128].abs()
        drop += x.shape[1] * 2.0 ** -13 * x.amax(1)[:, None] * y.amax(1)
    return a @ b.t(), a.abs() @ b.abs().t(), drop


def block_bound(K, S):
    """fp32: within a block at most 128 half steps of its sum, between blocks one per block, and the scales' product
    and its application one each."""
    return (min(K, 128) + blocks(K) + 4) * H * S


def layer64(X, R, w, b, eps):
    """(s, mean, rstd, y) and their bounds: s has one rounding for the residual; the mean's sum N of them; a deviation
    carries s', the mean's and its own; the variance twice the deviations' and its sum's; the root half the
    variance's, and six more for eps, the quotient and the root itself."""
    N = X.shape[1]
    s = X.double() if R is None else X.double() + R.double()
    mean = s.mean(1, keepdim=True)
    d = s - mean
    var = d.square().mean(1, keepdim=True)
    rstd = (var + eps).rsqrt()
    es = (0.0 if R is None else H) * s.abs()
    em = (N + 3) * H * s.abs().mean(1, keepdim=True)
    ed = es + em + H * (d.abs() + em)
    ev = (2 * d.abs() * ed + ed.square()).mean(1, keepdim=True) + (N + 4) * H * var
    er = 1.1 * ev / (2 * (var + eps)) + 6 * H
    y = d * rstd * w.double() + (0.0 if b is None else b.double())
    ey = w.double().abs() * rstd * (ed * (1 + er) + d.abs() * er) + 4 * H * (d * rstd * w.double()).abs() + H * y.abs()
    return (s, es), (mean[:, 0], em[:, 0]), (rstd[:, 0], (er * rstd)[:, 0]), (y, ey)


def layer_grad64(dY, S, w, mean, rstd, dS):
    """(dx, dweight, dbias) and their bounds for the given fp32 mean and rstd."""
    M, N = dY.shape
    r = rstd.double()[:, None]
    dy, x = dY.double(), S.double() - mean.double()[:, None]
    xh, g = x * r, dy * w.double()
    mg, mgx = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    dx = r * (g - mg - xh * mgx)
    e = r * ((N + 4) * H * g.abs().mean(1, keepdim=True) + xh.abs() * (N + 8) * H * (g * xh).abs().mean(1, keepdim=True)
             + 6 * H * (g.abs() + mg.abs() + (xh * mgx).abs())) + 2 * H * dx.abs()
    if dS is not None:
        dx = dx + dS.double()
        e = e + H * dx.abs()
    terms = (dy * xh).abs().sum(0)
    return (dx, e), ((dy * xh).sum(0), (M + 5) * H * terms), (dy.sum(0), (M + 2) * H * dy.abs().sum(0))


def rounded(bound, ref, dtype):
    """A bound with the rounding to dtype's format."""
    return bound + U[dtype] * (ref.abs() + bound) + TINY[dtype]


def e4m3(*shape, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * 60).clamp(-448, 448).to(F8)
