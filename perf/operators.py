"""The operators around a linear layer's training and serving, as cases to measure: layer norm with its backward, the
linear product in 8-bit floating point with a scale for each block of 128, and the orthogonalised update of a weight.

``run`` computes a case in its plain form (elementary torch operations in 32 bits) or, where ``own`` is true, through
the entry points of ``offload_streamed_gb300.tiled_linear``.  ``exact`` computes it in 64 bits from the definition.
"""
import math

import torch

own = False

BF16, F16, F32, F64 = torch.bfloat16, torch.float16, torch.float32, torch.float64
DTYPES = {"bf16": BF16, "fp16": F16, "fp32": F32}
EPS = 1e-5                          # layer norm's
NS = (3.4445, -4.7750, 2.0315)      # the quintic's coefficients
NS_STEPS, NS_EPS = 5, 1e-7
BLOCK = 128


def listed():
    return [
        # The norm before the GPT-scale layer: T = K = 8192.
        {"name": "norm fwd 8192x8192", "op": "norm_fwd", "rows": 8192, "cols": 8192, "dtype": "bf16"},
        {"name": "norm bwd 8192x8192", "op": "norm_bwd", "rows": 8192, "cols": 8192, "dtype": "bf16"},
        # The norm before the 64K-hidden layer: few rows, very long ones.
        {"name": "norm bwd 2048x65536", "op": "norm_bwd", "rows": 2048, "cols": 65536, "dtype": "bf16"},
        # One token of the 1T-width layer: latency.
        {"name": "norm fwd 1x25600", "op": "norm_fwd", "rows": 1, "cols": 25600, "dtype": "bf16"},
        # Odd sizes in full precision: no row starts on a vector's boundary.
        {"name": "norm bwd 517x5003 fp32", "op": "norm_bwd", "rows": 517, "cols": 5003, "dtype": "fp32"},
        # Serving, one token through the whole GPT-scale layer: the bytes of the weight.
        {"name": "linear 1x8192x32768", "op": "linear", "T": 1, "K": 8192, "n": 32768},
        # Serving, a few tokens through the smoke test's layer: latency.
        {"name": "linear 16x1024x4096", "op": "linear", "T": 16, "K": 1024, "n": 4096},
        # One tile of the 64K-hidden layer, forward: a long reduction.
        {"name": "linear 2048x65536x16384", "op": "linear", "T": 2048, "K": 65536, "n": 16384},
        # A training step of one tile of the GPT-scale layer, its weight in 8 bits anew.
        {"name": "step 8192x8192x4096", "op": "step", "T": 8192, "K": 8192, "n": 4096},
        # Small tiles of odd sizes, updated together.
        {"name": "orthogonal 4x200x520", "op": "orthogonal", "batch": 4, "rows": 200, "cols": 520, "dtype": "fp32"},
        # The smoke test's layer.
        {"name": "orthogonal 1024x4096", "op": "orthogonal", "batch": 1, "rows": 1024, "cols": 4096, "dtype": "bf16"},
        # Two tiles of the GPT-scale layer.
        {"name": "orthogonal 2x8192x4096", "op": "orthogonal", "batch": 2, "rows": 8192, "cols": 4096, "dtype": "bf16"},
    ]


def draw(rng):
    def size(lo, hi):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return max(lo, min(hi, v if rng.random() < 0.5 else (v + 63) // 64 * 64))

    while True:
        op = rng.choice(["norm_fwd", "norm_bwd", "linear", "step", "orthogonal"])
        if op in ("norm_fwd", "norm_bwd"):
            c = {"op": op, "rows": size(1, 32768), "cols": size(16, 65536), "dtype": rng.choice(["bf16", "fp16", "fp32"])}
            if c["rows"] * c["cols"] * (2 if c["dtype"] == "fp32" else 1) <= 2048 * 65536:
                return c
        elif op in ("linear", "step"):
            c = {"op": op, "T": size(1, 8192), "K": size(64, 32768), "n": size(64, 32768)}
            if 8192 <= c["T"] * c["K"] * c["n"] <= 8192 * 8192 * 4096:
                return c
        else:
            c = {"op": op, "batch": rng.choice([1, 1, 2, 3, 8]), "rows": size(32, 8192), "cols": size(32, 8192),
                 "dtype": rng.choice(["bf16", "bf16", "fp32"])}
            if work(c)["flops"] <= work(listed()[-1])["flops"]:
                return c


def work(case):
    op = case["op"]
    if op == "norm_fwd":
        r, c, e = case["rows"], case["cols"], DTYPES[case["dtype"]].itemsize
        return {"bytes": 2 * r * c * e + 2 * c * e + 8 * r, "flops": 8 * r * c}
    if op == "norm_bwd":
        r, c, e = case["rows"], case["cols"], DTYPES[case["dtype"]].itemsize
        return {"bytes": 3 * r * c * e + c * e + 8 * c + 8 * r, "flops": 14 * r * c}
    if op == "linear":
        T, K, n = case["T"], case["K"], case["n"]
        return {"bytes": 2 * T * K + K * n + 2 * T * n, "flops": 2 * T * K * n}
    if op == "step":  # reads x, w, dy; writes y, dx, dw
        T, K, n = case["T"], case["K"], case["n"]
        return {"bytes": 2 * (2 * T * K + 2 * K * n + 2 * T * n), "flops": 6 * T * K * n}
    b, r, c = case["batch"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
    return {"bytes": b * r * c * (DTYPES[case["dtype"]].itemsize + 2),
            "flops": b * NS_STEPS * (r * (r + 1) * c + r * r * (r + 1) + 2 * r * r * c)}


# ---- inputs --------------------------------------------------------------------------------------------------------

def _padded(rows, cols, dtype):
    """[rows, cols] whose rows start on 16-byte boundaries."""
    per = 16 // dtype.itemsize
    return torch.empty(rows, (cols + per - 1) // per * per, dtype=dtype, device="cuda")[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 11)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=F32)

    op, s = case["op"], {"op": case["op"]}
    if op in ("norm_fwd", "norm_bwd"):
        # residual-stream rows: a mean, a scale of their own, a few large channels
        r, c, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
        loud = 1 + 8 * (torch.rand(c, generator=g, device="cuda") < 0.01)
        s["x"] = (normal(r, c).mul_(loud).mul_(torch.exp(0.3 * normal(r, 1))).add_(0.2 * normal(r, 1))).to(dt)
        s["weight"] = (1 + 0.1 * normal(c)).to(dt)
        s["bias"] = (0.1 * normal(c)).to(dt)
        if op == "norm_bwd":
            s["dy"] = (0.01 * normal(r, c).mul_(torch.exp(0.5 * normal(r, 1)))).to(dt)
            xf = s["x"].float()
            s["mean"] = xf.mean(1)
            s["rstd"] = torch.rsqrt(xf.var(1, unbiased=False) + EPS)
        return s
    if op in ("linear", "step"):
        # activations after a norm (some channels larger), weights N(0, 1/K), gradients with scales of their own
        T, K, n = case["T"], case["K"], case["n"]
        s["x"] = normal(T, K).mul_(torch.exp(0.5 * normal(K))).to(BF16)
        w = normal(K, n).mul_(1 / math.sqrt(K)).to(BF16)
        if op == "linear":
            q, s["ws"] = _quantize(w, BLOCK, BLOCK)
            s["wq"] = _padded(K, n, torch.float8_e4m3fn)
            s["wq"].copy_(q)
        else:
            s["w"] = w
            s["dy"] = (0.01 * normal(T, n).mul_(torch.exp(0.5 * normal(T, 1)))).to(BF16)
        return s
    # a momentum: a few strong directions in noise whose columns differ in size
    b, r, c = case["batch"], case["rows"], case["cols"]
    k = max(1, min(r, c) // 64)
    m = normal(b, r, c).mul_(torch.exp(0.3 * normal(b, 1, c)))
    m += torch.bmm(normal(b, r, k), normal(b, k, c)).mul_(1 / math.sqrt(k))
    s["g"] = m.mul_(1e-3).to(DTYPES[case["dtype"]])
    return s


# ---- the plain forms -----------------------------------------------------------------------------------------------

def _blocks(x, br, bc):
    """x, padded with zeros, as [row blocks, br, column blocks, bc]."""
    r, c = x.shape
    x = torch.nn.functional.pad(x, (0, -c % bc, 0, -r % br))
    return x.reshape(x.shape[0] // br, br, x.shape[1] // bc, bc)


def _spread(v, br, bc, r, c):
    """One value a block, at each of the block's elements."""
    return v.repeat_interleave(br, 0)[:r].repeat_interleave(bc, 1)[:, :c]


def _pow2(e):
    """2^e for whole e in -127..127, exactly: written as bits, since pow() is rounded."""
    return torch.where(e > -127, (e + 127) << 23, 1 << 22).to(torch.int32).view(F32)


def _quantize(x, br, bc):
    """(q, scale): 8-bit e4m3 values and, for each br x bc block, the byte e + 127 of the least 2^e with
    amax <= 448 * 2^e (127 where the block is zero)."""
    x = x.float()
    amax = _blocks(x, br, bc).abs().amax((1, 3))
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(-127, 127)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    q = (x * _spread(_pow2(-e), br, bc, *x.shape)).to(torch.float8_e4m3fn)
    return q, (e + 127).to(torch.uint8)


def _values(q, scale, br, bc):
    return q.float() * _spread(_pow2(scale.int() - 127), br, bc, *q.shape)


def _rounded(x, br, bc):
    return _values(*_quantize(x, br, bc), br, bc)


def _norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = torch.rsqrt((d * d).mean(1, keepdim=True) + EPS)
    y = d * rstd * s["weight"].float() + s["bias"].float()
    return y.to(s["x"].dtype), mean[:, 0], rstd[:, 0]


def _norm_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    rstd = s["rstd"][:, None]
    xh = (x - s["mean"][:, None]) * rstd
    g = dy * s["weight"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx.to(s["x"].dtype), (dy * xh).sum(0), dy.sum(0)


def _linear(s):
    return (_rounded(s["x"], 1, BLOCK) @ _values(s["wq"], s["ws"], BLOCK, BLOCK)).to(BF16)


def _step(s):
    w = _rounded(s["w"], BLOCK, BLOCK)
    y = (_rounded(s["x"], 1, BLOCK) @ w).to(BF16)
    dx = (_rounded(s["dy"], 1, BLOCK) @ w.T).to(BF16)
    dw = (_rounded(s["x"], BLOCK, 1).T @ _rounded(s["dy"], BLOCK, 1)).to(BF16)
    return y, dx, dw


def _orthogonal(s):
    a, b, c = NS
    x = s["g"].float()
    tall = x.shape[1] > x.shape[2]
    x = x.mT if tall else x
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    for _ in range(NS_STEPS):
        p = x @ x.mT
        x = a * x + (b * p + c * (p @ p)) @ x
    return (x.mT if tall else x).to(BF16).contiguous()


def run(state):
    op = state["op"]
    if not own:
        return {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "linear": _linear, "step": _step,
                "orthogonal": _orthogonal}[op](state)
    from offload_streamed_gb300 import tiled_linear as tl
    if op == "norm_fwd":
        return tl.layer_norm(state["x"], state["weight"], state["bias"], EPS)
    if op == "norm_bwd":
        return tl.layer_norm_backward(state["dy"], state["x"], state["mean"], state["rstd"], state["weight"])
    if op == "linear":
        return tl.fp8_linear(state["x"], state["wq"], state["ws"])
    if op == "step":
        wq, ws = tl.fp8_quantize(state["w"], "tile")
        y = tl.fp8_linear(state["x"], wq, ws)
        dx, dw = tl.fp8_linear_backward(state["x"], state["dy"], wq, ws)
        return y, dx, dw
    return tl.orthogonalize(state["g"], steps=NS_STEPS, coefficients=NS, eps=NS_EPS)


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------

def _pow64(e):
    return ((e.to(torch.int64) + 1023) << 52).view(F64)


def _held64(x, br, bc):
    """The values that x's 8-bit form stands for: each v becomes the multiple of 2^k nearest to it (ties to the even
    one), where 2^k is the spacing of the 4-bit significands at |v| for the block's scale."""
    r, c = x.shape
    v = x.to(F64)
    top = torch.zeros(-(-r // br), -(-c // bc), dtype=F64, device=x.device)
    for i in range(br):       # the blocks' largest magnitudes, one row and one column of each block at a time
        rows = v[i::br].abs()
        if rows.shape[0]:
            rows = torch.nn.functional.pad(rows, (0, -c % bc)).reshape(rows.shape[0], -1, bc).amax(2)
            top[:rows.shape[0]] = torch.maximum(top[:rows.shape[0]], rows)
    e = torch.ceil(torch.log2(top.clamp_min(2.0 ** -400) / 448))
    e = torch.where(top > 448 * _pow64(e), e + 1, torch.where(top <= 448 * _pow64(e - 1), e - 1, e)).clamp(-127, 127)
    unit = _pow64(e)[torch.arange(r, device=x.device) // br][:, torch.arange(c, device=x.device) // bc]
    size = torch.frexp(v.abs() / unit).exponent - 1
    step = unit * _pow64(size.clamp_min(-6) - 3)
    return torch.round(v / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_fwd":
        x = s["x"].to(F64)
        n = x.shape[1]
        mean = x.sum(1) / n
        var = (x * x).sum(1) / n - mean * mean
        rstd = 1 / torch.sqrt(var + EPS)
        return (x - mean[:, None]) * (rstd[:, None] * s["weight"].to(F64)) + s["bias"].to(F64), mean, rstd
    if op == "norm_bwd":
        x, dy, w = s["x"].to(F64), s["dy"].to(F64), s["weight"].to(F64)
        m, r, n = s["mean"].to(F64), s["rstd"].to(F64), x.shape[1]
        x = (x - m[:, None]) * r[:, None]
        dw, db = torch.einsum("tc,tc->c", dy, x), dy.sum(0)
        c1, c2 = dy @ w / n, torch.einsum("tc,tc,c->t", dy, x, w) / n
        return (dy * w - c1[:, None] - x * c2[:, None]) * r[:, None], dw, db
    if op == "linear":
        scale = _pow64(s["ws"].int() - 127)
        K, n = s["wq"].shape
        w = s["wq"].to(F64) * scale[torch.arange(K, device="cuda") // BLOCK][:, torch.arange(n, device="cuda") // BLOCK]
        return _held64(s["x"], 1, BLOCK) @ w
    if op == "step":
        w = _held64(s["w"], BLOCK, BLOCK)
        y, dx = _held64(s["x"], 1, BLOCK) @ w, _held64(s["dy"], 1, BLOCK) @ w.T
        return y, dx, _held64(s["x"].T, 1, BLOCK) @ _held64(s["dy"].T, 1, BLOCK).T
    x = s["g"].to(F64)
    x = x / (torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True) + NS_EPS)
    a, b, c = NS
    for _ in range(NS_STEPS):   # on whichever side is short, written for the long one's products
        if x.shape[1] <= x.shape[2]:
            p = torch.einsum("bik,bjk->bij", x, x)
            x = a * x + b * (p @ x) + c * (p @ (p @ x))
        else:
            p = torch.einsum("bki,bkj->bij", x, x)
            x = a * x + b * (x @ p) + c * ((x @ p) @ p)
    return x
