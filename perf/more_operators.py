"""The operators of a feed-forward block in plain torch and through the package: gated projections
(two products of the same rows, the activation of one times the other; forward and backward), layer
norms with the residual's addition (16- and 32-bit output or 8 bits with a scale per 128 columns;
forward and backward), and products of 8-bit operands with a scale per block of 128.

`run` computes one pass of one operator: with `own` false in elementary torch operations, in 32 bits
with one rounding at the end; with `own` true through the package's entry points."""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
SCALE_MIN = 2.0 ** -100
BLOCK = 128
EPS = 1e-5
ACTS = ("silu", "silu", "gelu_tanh", "gelu", "relu", "none")
WORKSPACE = 256 << 20
WORKSPACE_BWD = 640 << 20


def listed():
    return [
        # One token through a block's gate and up projections while generating: the weights' bytes count.
        {"name": "gated_token", "op": "gated", "M": 1, "N": 14336, "K": 4096, "dtype": "bf16", "act": "silu",
         "bias": False, "preact": False},
        # A small fp32 block, pre-activations kept for its backward pass.
        {"name": "gated_small_f32", "op": "gated", "M": 512, "N": 512, "K": 512, "dtype": "f32",
         "act": "gelu_tanh", "bias": True, "preact": True},
        # The forward pass of a training step: a long batch, pre-activations kept.
        {"name": "gated_train", "op": "gated", "M": 8192, "N": 8192, "K": 4096, "dtype": "bf16", "act": "silu",
         "bias": False, "preact": True},
        # The backward pass of a block of ordinary size.
        {"name": "gated_backward", "op": "gated_bwd", "M": 4096, "N": 8192, "K": 4096, "dtype": "bf16",
         "act": "silu", "bias": False},
        # A ragged backward pass of few rows, with the biases' gradients.
        {"name": "gated_backward_ragged", "op": "gated_bwd", "M": 1000, "N": 2744, "K": 1032, "dtype": "f16",
         "act": "gelu_tanh", "bias": True},
        # A few sequences' next tokens through an 8-bit projection, activations quantized on the way.
        {"name": "f8_block_tokens", "op": "f8_block", "M": 16, "N": 4096, "K": 4096, "dtype": "bf16",
         "act": "none", "bias": False, "residual": True, "quant": True},
        # A long prompt through an 8-bit projection whose operand the norm has written.
        {"name": "f8_block_prompt", "op": "f8_block", "M": 4096, "N": 4096, "K": 4096, "dtype": "bf16",
         "act": "none", "bias": False, "residual": False, "quant": False},
        # A weight's gradient from a batch in 8 bits: both operands quantized along the batch.
        {"name": "f8_block_weight_grad", "op": "f8_block_grad", "M": 2048, "N": 4096, "K": 8192, "dtype": "bf16"},
        # The norm before a projection for one token, straight to the product's 8-bit operand.
        {"name": "layer_norm_token_f8", "op": "norm", "M": 1, "N": 4096, "dtype": "bf16", "residual": True,
         "bias": True, "f8": True},
        # The norm of a training step's forward pass: sum, mean and reciprocal root kept.
        {"name": "layer_norm_train", "op": "norm", "M": 16384, "N": 4096, "dtype": "bf16", "residual": True,
         "bias": True, "f8": False},
        # Its backward pass, the residual's gradient added.
        {"name": "layer_norm_backward", "op": "norm_bwd", "M": 16384, "N": 4096, "dtype": "bf16",
         "residual": True, "bias": True},
        # The same for a ragged fp16 row length and few rows.
        {"name": "layer_norm_backward_ragged", "op": "norm_bwd", "M": 1000, "N": 2999, "dtype": "f16",
         "residual": False, "bias": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_bwd", "gated_bwd", "f8_block", "f8_block", "f8_block_grad", "norm",
                     "norm_bwd"])
    M = _log_int(rng, 1, 16384)
    c = {"op": op, "M": M}
    if op in ("norm", "norm_bwd"):
        c.update(N=_log_int(rng, 64, 8192), dtype=rng.choice(["bf16", "f16", "f32"]),
                 residual=rng.random() < 0.6, bias=rng.random() < 0.7)
        if op == "norm":
            c["f8"] = rng.random() < 0.5
        return c
    c.update(N=_log_int(rng, 64, 8192), K=_log_int(rng, 64, 4104))
    if op == "f8_block_grad":
        c.update(M=_log_int(rng, 64, 4104), N=_log_int(rng, 64, 4104), K=M, dtype=rng.choice(["bf16", "f16", "f32"]))
        return c
    c["act"] = rng.choice(ACTS)
    c["bias"] = rng.random() < 0.5
    if op == "f8_block":
        c.update(dtype=rng.choice(["bf16", "f16", "f32"]), residual=rng.random() < 0.5, quant=rng.random() < 0.5)
        return c
    c["dtype"] = rng.choice(["bf16", "bf16", "f16", "f16", "f32"])
    if c["dtype"] == "f32":  # the fp32 matrix rate is a sixteenth of the 16-bit one
        c["M"] = min(M, 2048)
        c["N"] = min(c["N"], 4104)
    c["M"] = min(c["M"], 8192 if op == "gated" else 4096)
    if op == "gated":
        c["preact"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------------------------------ inputs

def _matrix(rows, cols, dtype):
    """A row-major matrix whose row pitch is a multiple of 16 bytes, as the framework asks."""
    per16 = 16 // torch.empty((), dtype=dtype).element_size()
    pitch = (cols + per16 - 1) // per16 * per16
    return torch.zeros((rows, pitch), dtype=dtype, device="cuda")[:, :cols]


def _normal(gen, rows, cols, dtype, scale=1.0):
    m = _matrix(rows, cols, dtype)
    m.copy_(torch.randn((rows, cols), generator=gen, device="cuda") * scale)
    return m


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def _scales(rows, cols):
    """A scale per row and block of columns, rows next to each other in memory."""
    return torch.empty((cols, rows), device="cuda").t()


def _to_f8(x, rows):
    """x in 8 bits with a scale for every `rows` x 128 of it: (codes, scales)."""
    r, c = x.shape
    rb, cb = (r + rows - 1) // rows, _blocks(c)
    whole = torch.nn.functional.pad(x, (0, cb * BLOCK - c, 0, rb * rows - r)).view(rb, rows, cb, BLOCK)
    amax = whole.abs().amax(dim=(1, 3))
    # a division by a tensor: torch multiplies by a rounded reciprocal where the divisor is a plain number
    scale = (amax / torch.full_like(amax, F8_MAX)).clamp_min(SCALE_MIN)
    # The quotient in 64 bits, rounded once: 32 bits put some next to a border between two codes on it.
    v = whole.double() / scale.double()[:, None, :, None]
    step = torch.ldexp(torch.ones_like(v), (torch.frexp(v).exponent - 1).clamp_min(-6) - 3)
    v = ((v / step).round() * step).clamp(-F8_MAX, F8_MAX).reshape(rb * rows, cb * BLOCK)[:r, :c]
    q = _matrix(r, c, F8)
    q.copy_(v.to(F8))
    return q, scale


def _from_f8(q, scale, rows):
    """The values that codes and scales stand for."""
    s = scale.repeat_interleave(rows, dim=0)[: q.shape[0]].repeat_interleave(BLOCK, dim=1)[:, : q.shape[1]]
    return q.to(scale.dtype) * s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, M, N = case["op"], case["M"], case["N"]
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    s["workspace"] = torch.empty(WORKSPACE_BWD if op == "gated_bwd" else WORKSPACE, dtype=torch.uint8,
                                 device="cuda")
    if op in ("norm", "norm_bwd"):
        # Hidden states with a few large channels and a common offset, as residual streams have.
        ch = torch.ones(N, device="cuda")
        ch[:: max(1, N // 8)] = 8.0
        s["X"] = _matrix(M, N, dt)
        s["X"].copy_(torch.randn((M, N), generator=gen, device="cuda") * ch + 0.25)
        s["weight"] = 1.0 + 0.2 * torch.randn(N, generator=gen, device="cuda")
        s["R"] = _normal(gen, M, N, dt, ch) if case["residual"] else None
        if op == "norm":
            s["bias"] = 0.1 * torch.randn(N, generator=gen, device="cuda") if case["bias"] else None
            s["Y"] = _matrix(M, N, F8 if case["f8"] else dt)
            s["S"] = _matrix(M, N, dt) if case["residual"] else None
            s["scale"] = _scales(M, _blocks(N)) if case["f8"] else None
            s["mean"] = None if case["f8"] else torch.empty(M, device="cuda")
            s["rstd"] = None if case["f8"] else torch.empty(M, device="cuda")
        else:
            # X stands for the forward pass's stored sum, R for the gradient that the residual brings.
            s["dY"] = _normal(gen, M, N, dt, 0.1)
            if s["R"] is not None:
                s["R"].mul_(0.1)
            x = s["X"].float()
            s["mean"] = x.mean(dim=1)
            s["rstd"] = (x.var(dim=1, unbiased=False) + EPS).rsqrt()
            s["dX"] = _matrix(M, N, dt)
            s["dweight"] = torch.empty(N, device="cuda")
            s["dbias"] = torch.empty(N, device="cuda") if case["bias"] else None
        return s
    K = case["K"]
    if op == "f8_block_grad":
        s["X"], s["dZ"] = _normal(gen, K, M, dt), _normal(gen, K, N, dt, 0.1)
        s["A"], s["scale_a"] = _matrix(M, K, F8), _scales(M, _blocks(K))
        s["B"], s["scale_b"] = _matrix(N, K, F8), _scales(N, _blocks(K))
        s["C"] = _matrix(M, N, dt)
        return s
    if op == "f8_block":
        s["bias"] = 0.1 * torch.randn(N, generator=gen, device="cuda") if case["bias"] else None
        # Activations whose size differs from channel to channel, as the blocks' scales are for.
        ch = 1.0 + 7.0 * torch.rand(K, generator=gen, device="cuda").pow(8)
        x = _normal(gen, M, K, dt, ch)
        s["B"], s["scale_b"] = _to_f8(torch.randn((N, K), generator=gen, device="cuda") / math.sqrt(K), BLOCK)
        if case["quant"]:
            s["X"] = x
            s["A"], s["scale_a"] = _matrix(M, K, F8), _scales(M, _blocks(K))
        else:
            s["A"], scale = _to_f8(x.float(), 1)
            s["scale_a"] = _scales(M, _blocks(K)).copy_(scale)
        s["R"] = _normal(gen, M, N, dt) if case["residual"] else None
        s["C"] = _matrix(M, N, dt)
        return s
    s["A"] = _normal(gen, M, K, dt)
    s["Bg"] = _normal(gen, K, N, dt, 1.0 / math.sqrt(K))
    s["Bu"] = _normal(gen, K, N, dt, 1.0 / math.sqrt(K))
    if op == "gated_bwd":
        s["dC"] = _normal(gen, M, N, dt, 0.1)
        s["G"], s["U"] = _normal(gen, M, N, dt), _normal(gen, M, N, dt)
        s["dA"], s["dBg"], s["dBu"] = _matrix(M, K, dt), _matrix(K, N, dt), _matrix(K, N, dt)
        s["dbias_g"] = torch.empty(N, device="cuda") if case["bias"] else None
        s["dbias_u"] = torch.empty(N, device="cuda") if case["bias"] else None
        return s
    s["bias_g"] = 0.1 * torch.randn(N, generator=gen, device="cuda") if case["bias"] else None
    s["bias_u"] = 0.1 * torch.randn(N, generator=gen, device="cuda") if case["bias"] else None
    s["C"] = _matrix(M, N, dt)
    s["G"] = _matrix(M, N, dt) if case["preact"] else None
    s["U"] = _matrix(M, N, dt) if case["preact"] else None
    return s


# --------------------------------------------------------------------------------------- plain form

def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return torch.ones_like(z)


def _plain(s):
    c, dt = s["case"], DTYPES[s["case"]["dtype"]]
    op = c["op"]
    if op == "gated":
        a = s["A"].float()
        g, u = a @ s["Bg"].float(), a @ s["Bu"].float()
        if c["bias"]:
            g, u = g + s["bias_g"], u + s["bias_u"]
        out = {"C": (_act(g, c["act"]) * u).to(dt)}
        if c["preact"]:
            out["G"], out["U"] = g.to(dt), u.to(dt)
        return out
    if op == "gated_bwd":
        dc, g, u = s["dC"].float(), s["G"].float(), s["U"].float()
        dg, du = dc * u * _act_grad(g, c["act"]), dc * _act(g, c["act"])
        at = s["A"].float().t()
        out = {"dA": (dg @ s["Bg"].float().t() + du @ s["Bu"].float().t()).to(dt), "dBg": (at @ dg).to(dt),
               "dBu": (at @ du).to(dt)}
        if c["bias"]:
            out["dbias_g"], out["dbias_u"] = dg.sum(dim=0), du.sum(dim=0)
        return out
    if op == "f8_block_grad":
        qa, sa = _to_f8(s["X"].float().t(), 1)
        qb, sb = _to_f8(s["dZ"].float().t(), 1)
        return {"C": (_from_f8(qa, sa, 1) @ _from_f8(qb, sb, 1).t()).to(dt)}
    if op == "f8_block":
        a, sa = _to_f8(s["X"].float(), 1) if c["quant"] else (s["A"], s["scale_a"])
        z = _from_f8(a, sa, 1) @ _from_f8(s["B"], s["scale_b"], BLOCK).t()
        if s["bias"] is not None:
            z = z + s["bias"]
        y = _act(z, c["act"])
        if s["R"] is not None:
            y = y + s["R"].float()
        return {"C": y.to(dt)}
    x, w = s["X"].float(), s["weight"]
    if op == "norm":
        if s["R"] is not None:
            x = x + s["R"].float()
        mean = x.mean(dim=1, keepdim=True)
        d = x - mean
        rstd = (d.square().mean(dim=1, keepdim=True) + EPS).rsqrt()
        y = d * rstd * w
        if s["bias"] is not None:
            y = y + s["bias"]
        out = {}
        if c["f8"]:
            out["Y"], out["scale"] = _to_f8(y, 1)
        else:
            out["Y"], out["mean"], out["rstd"] = y.to(dt), mean[:, 0], rstd[:, 0]
        if s["R"] is not None:
            out["S"] = x.to(dt)
        return out
    dy, rstd = s["dY"].float(), s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    g = dy * w
    dx = rstd * (g - g.mean(dim=1, keepdim=True) - xh * (g * xh).mean(dim=1, keepdim=True))
    if s["R"] is not None:
        dx = dx + s["R"].float()
    out = {"dX": dx.to(dt), "dweight": (dy * xh).sum(dim=0)}
    if c["bias"]:
        out["dbias"] = dy.sum(dim=0)
    return out


# ------------------------------------------------------------------------------------ the package

def _own(s):
    import dense_gemm_matrix_amd as dg
    c = s["case"]
    op = c["op"]
    if op == "gated":
        dg.gemm_gated(s["A"], s["Bg"], s["Bu"], s["C"], bias_g=s["bias_g"], bias_u=s["bias_u"], act=c["act"],
                      gate=s["G"], up=s["U"], workspace=s["workspace"])
        return {"C": s["C"], "G": s["G"], "U": s["U"]} if c["preact"] else {"C": s["C"]}
    if op == "gated_bwd":
        dg.gemm_gated_bwd(s["A"], s["Bg"], s["Bu"], s["dC"], s["G"], s["U"], act=c["act"], dA=s["dA"],
                          dBg=s["dBg"], dBu=s["dBu"], dbias_g=s["dbias_g"], dbias_u=s["dbias_u"],
                          workspace=s["workspace"])
        out = {"dA": s["dA"], "dBg": s["dBg"], "dBu": s["dBu"]}
        if c["bias"]:
            out["dbias_g"], out["dbias_u"] = s["dbias_g"], s["dbias_u"]
        return out
    if op == "f8_block_grad":
        dg.quant_f8_block(s["X"], s["A"], s["scale_a"], transpose=True)
        dg.quant_f8_block(s["dZ"], s["B"], s["scale_b"], transpose=True)
        dg.gemm_f8_block(s["A"], s["B"], s["C"], s["scale_a"], s["scale_b"], workspace=s["workspace"])
        return {"C": s["C"]}
    if op == "f8_block":
        if c["quant"]:
            dg.quant_f8_block(s["X"], s["A"], s["scale_a"])
        dg.gemm_f8_block(s["A"], s["B"], s["C"], s["scale_a"], s["scale_b"], bias=s["bias"], act=c["act"],
                         residual=s["R"], workspace=s["workspace"])
        return {"C": s["C"]}
    if op == "norm":
        dg.layernorm(s["X"], s["weight"], s["bias"], s["Y"], residual=s["R"], total=s["S"], scale=s["scale"],
                     mean=s["mean"], rstd=s["rstd"], eps=EPS)
        out = {"Y": s["Y"]}
        for k in ("scale", "S", "mean", "rstd"):
            if s[k] is not None:
                out[k] = s[k]
        return out
    dg.layernorm_bwd(s["dY"], s["X"], s["weight"], s["mean"], s["rstd"], s["dX"], dtotal=s["R"],
                     dweight=s["dweight"], dbias=s["dbias"], workspace=s["workspace"])
    out = {"dX": s["dX"], "dweight": s["dweight"]}
    if c["bias"]:
        out["dbias"] = s["dbias"]
    return out


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------------------- the least work

def work(case):
    op, M, N = case["op"], case["M"], case["N"]
    es = 4 if case["dtype"] == "f32" else 2
    if op == "norm":
        b = M * N * es * (3 if case["residual"] else 1) + (8 if case["bias"] else 4) * N
        b += M * N + 4 * M * _blocks(N) if case["f8"] else M * N * es + 8 * M
        return {"bytes": b, "flops": 9 * M * N}
    if op == "norm_bwd":
        return {"bytes": M * N * es * (4 if case["residual"] else 3) + 8 * M + (12 if case["bias"] else 8) * N,
                "flops": 14 * M * N}
    K = case["K"]
    if op == "f8_block_grad":
        return {"bytes": (K * M + K * N + M * N) * es, "flops": 2 * M * N * K}
    if op == "f8_block":
        mn = 1 + bool(case["residual"])
        a = M * K * es if case["quant"] else M * K + 4 * M * _blocks(K)
        return {"bytes": a + N * K + 4 * _blocks(N) * _blocks(K) + mn * M * N * es + (4 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    bias = 8 * N if case["bias"] else 0
    if op == "gated":
        return {"bytes": (M * K + 2 * K * N + (3 if case["preact"] else 1) * M * N) * es + bias,
                "flops": 4 * M * N * K}
    return {"bytes": (2 * M * K + 4 * K * N + 3 * M * N) * es + bias, "flops": 8 * M * N * K}


# ---------------------------------------------------------------------- the definitions in 64 bits

def _e4m3_blocks(y):
    """Rows in 8 bits, a scale per 128 columns: the scales, which are values of 32 bits, and the quotients by
    them rounded to the nearest value with three fraction bits (ties to even), steps no finer than 2^-9."""
    n = y.shape[1]
    part = torch.zeros((y.shape[0], _blocks(n) * BLOCK), dtype=y.dtype, device=y.device)
    part[:, :n] = y
    part = part.view(y.shape[0], -1, BLOCK)
    scale = torch.clamp(part.abs().max(dim=2).values / F8_MAX, min=SCALE_MIN).float().double()
    v = part / scale.unsqueeze(2)
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(v.abs().clamp_min(1e-300))), min=-6.0) - 3.0)
    return (torch.round(v / step) * step), scale


def _values(codes, scale, n):
    return (codes * scale.unsqueeze(2)).reshape(codes.shape[0], -1)[:, :n]


def _value64(act):
    tau = lambda z: math.sqrt(2.0 / math.pi) * z * (1.0 + 0.044715 * z ** 2)  # noqa: E731
    return {"none": lambda z: z, "relu": lambda z: z.clamp_min(0.0),
            "gelu": lambda z: z * 0.5 * torch.erfc(-z / math.sqrt(2.0)),
            "gelu_tanh": lambda z: z * torch.sigmoid(2.0 * tau(z)), "silu": lambda z: z * torch.sigmoid(z)}[act]


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and k != "workspace"}
    op = case["op"]
    if op == "gated":
        both = torch.mm(d["A"], torch.cat([d["Bg"], d["Bu"]], dim=1))
        if case["bias"]:
            both += torch.cat([d["bias_g"], d["bias_u"]])
        g, u = both.chunk(2, dim=1)
        c = u * _value64(case["act"])(g)
        return {"C": c, "G": g, "U": u} if case["preact"] else {"C": c}
    if op == "gated_bwd":
        g, u = d["G"].clone().requires_grad_(True), d["U"].clone().requires_grad_(True)
        with torch.enable_grad():
            grads = torch.autograd.grad(_value64(case["act"])(g) * u, (g, u), d["dC"])
        both = torch.cat(grads, dim=1)
        if case["act"] == "relu":
            both = torch.cat([d["dC"] * d["U"] * (d["G"] > 0), d["dC"] * d["G"].clamp_min(0.0)], dim=1)
        n = case["N"]
        dw = torch.mm(d["A"].t(), both)
        out = {"dA": torch.mm(both, torch.cat([d["Bg"], d["Bu"]], dim=1).t()), "dBg": dw[:, :n], "dBu": dw[:, n:]}
        if case["bias"]:
            total = torch.ones(1, both.shape[0], dtype=both.dtype, device=both.device).mm(both)[0]
            out["dbias_g"], out["dbias_u"] = total[:n], total[n:]
        return out
    if op == "f8_block_grad":
        a, b = (_values(*_e4m3_blocks(d[k].t()), case["K"]) for k in ("X", "dZ"))
        return {"C": torch.mm(a, b.t())}
    if op == "f8_block":
        K, N = case["K"], case["N"]
        if case["quant"]:
            a = _values(*_e4m3_blocks(d["X"]), K)
        else:
            at = torch.arange(K, device="cuda") // BLOCK
            a = d["A"] * d["scale_a"][:, at]
        rows, cols = torch.arange(N, device="cuda") // BLOCK, torch.arange(K, device="cuda") // BLOCK
        z = torch.mm(a, (d["B"] * d["scale_b"][rows][:, cols]).t())
        if case["bias"]:
            z += d["bias"]
        c = _value64(case["act"])(z)
        return {"C": c + d["R"] if case["residual"] else c}
    if op == "norm":
        t = d["X"] + d["R"] if case["residual"] else d["X"]
        n = case["N"]
        mean = t.sum(dim=1) / n
        var = (t * t).sum(dim=1) / n - mean * mean
        root = torch.sqrt(var + EPS)
        y = (t - mean.unsqueeze(1)) / root.unsqueeze(1) * d["weight"]
        if case["bias"]:
            y = y + d["bias"]
        out = {}
        if case["f8"]:
            codes, out["scale"] = _e4m3_blocks(y)
            out["Y"] = codes.reshape(codes.shape[0], -1)[:, :n]
        else:
            out["Y"], out["mean"], out["rstd"] = y, mean, 1.0 / root
        if case["residual"]:
            out["S"] = t
        return out
    # The gradient of sum(dY o ((x - mean) rstd w + b)), mean and rstd functions of x, their values as given.
    r, n = d["rstd"].unsqueeze(1), case["N"]
    t = d["X"] - d["mean"].unsqueeze(1)
    g = d["dY"] * d["weight"]
    dx = r * (g - g.sum(dim=1, keepdim=True) / n) - t * (r ** 3) * (g * t).sum(dim=1, keepdim=True) / n
    if case["residual"]:
        dx = dx + d["R"]
    out = {"dX": dx, "dweight": (d["dY"] * t * r).sum(dim=0)}
    if case["bias"]:
        out["dbias"] = d["dY"].sum(dim=0)
    return out
