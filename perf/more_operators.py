"""The operators of a linear layer whose weight depends on the row, as cases to measure: the router that sends tokens to
experts and sums their answers, the products grouped by expert with ragged sizes, and low-rank adapters of many requests
beside a shared projection; each with its backward pass.

``run`` computes a case in its plain form (elementary torch operations in 32 bits) or, where ``own`` is true, through
the entry points of ``offload_streamed_gb300.tiled_linear``.  ``exact`` computes it in 64 bits from the definition.
"""
import math

import torch

own = False

BF16, F16, F32, F64, I32 = torch.bfloat16, torch.float16, torch.float32, torch.float64, torch.int32
DTYPES = {"bf16": BF16, "fp16": F16, "fp32": F32}


def listed():
    return [
        # A prefill of many tokens over many small experts: the logits' bytes.
        {"name": "route 65536x256 top 8", "op": "route", "T": 65536, "E": 256, "k": 8, "dtype": "bf16", "normalize": True},
        # One decoding step of a small batch: latency.  Some experts are masked out.
        {"name": "route 32x128 top 4", "op": "route", "T": 32, "E": 128, "k": 4, "dtype": "fp32", "normalize": False},
        # The router's part of a training step, over all experts' probabilities.
        {"name": "route bwd 8192x64 top 2", "op": "route_bwd", "T": 8192, "E": 64, "k": 2, "dtype": "fp32", "normalize": False},
        # The experts' answers summed for the GPT-scale layer's tokens.
        {"name": "combine 8192x8192 top 2", "op": "combine", "T": 8192, "C": 8192, "k": 2, "dtype": "bf16"},
        # Its backward with many experts a token and odd sizes.
        {"name": "combine bwd 4099x1000 top 8", "op": "combine_bwd", "T": 4099, "C": 1000, "k": 8, "dtype": "fp16"},
        # Decoding, 16 tokens through 8 experts of a GPT-scale tile: the bytes of the experts that are met.
        {"name": "grouped 16x8192x4096 of 8", "op": "grouped", "T": 16, "k": 2, "E": 8, "K": 8192, "n": 4096,
         "gather": True, "dtype": "bf16"},
        # The GPT-scale tile as eight experts, tokens picked up where they lie.
        {"name": "grouped 8192x8192x4096 of 8", "op": "grouped", "T": 8192, "k": 2, "E": 8, "K": 8192, "n": 4096,
         "gather": True, "dtype": "bf16"},
        # A training step's backward: sixteen experts of a middling layer.
        {"name": "grouped bwd 8192x4096x4096 of 16", "op": "grouped_bwd", "T": 8192, "k": 2, "E": 16, "K": 4096, "n": 4096,
         "gather": True, "dtype": "bf16"},
        # Many small experts of odd sizes, rows in order already, some groups empty.
        {"name": "grouped bwd 2050x1000x520 of 64", "op": "grouped_bwd", "T": 2050, "k": 1, "E": 64, "K": 1000, "n": 520,
         "gather": False, "dtype": "fp16"},
        # Decoding: 32 requests, most with an adapter of their own.
        {"name": "adapters 32x8192x8192 rank 16 of 64", "op": "adapter", "T": 32, "K": 8192, "n": 8192, "r": 16, "R": 64,
         "runs": 1, "dtype": "bf16"},
        # Prefill: long requests beside a tile of the GPT-scale layer.
        {"name": "adapters 8192x8192x4096 rank 64 of 8", "op": "adapter", "T": 8192, "K": 8192, "n": 4096, "r": 64, "R": 8,
         "runs": 500, "dtype": "bf16"},
        # Training a few adapters at once beside the same tile.
        {"name": "adapters bwd 8192x8192x4096 rank 16 of 4", "op": "adapter_bwd", "T": 8192, "K": 8192, "n": 4096, "r": 16,
         "R": 4, "runs": 1024, "dtype": "bf16"},
    ]


def draw(rng):
    def size(lo, hi, to=64):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return max(lo, min(hi, v if rng.random() < 0.5 else (v + to - 1) // to * to))

    most = max(work(c)["flops"] for c in listed())
    while True:
        op = rng.choice(["route", "route_bwd", "combine", "combine_bwd", "grouped", "grouped", "grouped_bwd", "adapter",
                         "adapter", "adapter_bwd"])
        if op in ("route", "route_bwd"):
            E = size(8, 512, 8)
            c = {"op": op, "T": size(1, 65536), "E": E, "k": rng.randint(1, min(8, E)),
                 "dtype": rng.choice(["bf16", "fp16", "fp32"]), "normalize": rng.random() < 0.5}
            if c["T"] * E <= 65536 * 256:
                return c
        elif op in ("combine", "combine_bwd"):
            c = {"op": op, "T": size(1, 16384), "C": size(16, 16384), "k": rng.randint(1, 8),
                 "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
            if c["T"] * c["C"] * c["k"] <= 8192 * 8192 * 2:
                return c
        elif op in ("grouped", "grouped_bwd"):
            k = rng.choice([1, 2, 2, 4])
            c = {"op": op, "T": size(1, 8192), "k": k, "E": size(max(2, k), 128, 8), "K": size(64, 8192), "n": size(64, 8192),
                 "gather": rng.random() < 0.7, "dtype": rng.choice(["bf16", "bf16", "fp16"])}
            if c["E"] * c["K"] * c["n"] <= 8 * 8192 * 4096 and work(c)["flops"] <= most:
                return c
        else:
            c = {"op": op, "T": size(1, 8192), "K": size(64, 8192), "n": size(64, 8192), "r": rng.choice([4, 8, 16, 16, 32, 64, 128]),
                 "R": size(1, 64, 4), "runs": size(1, 1024), "dtype": rng.choice(["bf16", "bf16", "fp16"])}
            if c["T"] * max(c["K"], c["n"]) <= 8192 * 8192:
                return c


def work(case):
    op, e = case["op"], DTYPES[case["dtype"]].itemsize
    if op == "route":  # reads the logits; writes weights, ids, slots, rows and offsets
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * e + 16 * T * k + 4 * E + 4, "flops": T * E * (1 if case["normalize"] else 4) + 4 * T * k}
    if op == "route_bwd":  # reads the weights' gradients, the ids and the logits it needs; writes all logits' gradients
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * (k if case["normalize"] else E) * e + T * E * e + 8 * T * k, "flops": T * (k if case["normalize"] else E) * 5}
    if op == "combine":
        T, C, k = case["T"], case["C"], case["k"]
        return {"bytes": (k + 1) * T * C * e + 8 * T * k, "flops": 2 * k * T * C}
    if op == "combine_bwd":
        T, C, k = case["T"], case["C"], case["k"]
        return {"bytes": (2 * k + 1) * T * C * e + 12 * T * k, "flops": 3 * k * T * C}
    if op in ("grouped", "grouped_bwd"):
        T, k, E, K, n = (case[v] for v in ("T", "k", "E", "K", "n"))
        R, tokens = T * k, T if case["gather"] else T * k
        met = E * (1 - (1 - 1 / E) ** R)  # experts that some row goes to
        if op == "grouped":
            return {"bytes": int(e * (tokens * K + met * K * n + R * n)), "flops": 2 * R * K * n}
        return {"bytes": int(e * (tokens * K + R * n + met * K * n + R * K + E * K * n)), "flops": 4 * R * K * n}
    T, K, n, r, R = (case[v] for v in ("T", "K", "n", "r", "R"))
    met = R * (1 - (1 - 1 / R) ** max(1, T // case["runs"])) if R > 1 else 1
    if op == "adapter":  # reads x, base, A and B; writes y and h
        return {"bytes": int(e * (T * K + 2 * T * n + met * r * (K + n) + T * r)), "flops": 2 * T * r * (K + n)}
    # reads x, h, dy, the other part of dx, A and B; writes dx, dA and dB
    return {"bytes": int(e * (3 * T * K + T * n + (met + R) * r * (K + n) + T * r)), "flops": 4 * T * r * (K + n)}


# ---- inputs --------------------------------------------------------------------------------------------------------

def _rows16(*shape, dtype=BF16):
    """An empty tensor whose rows start on 16-byte boundaries."""
    per = 16 // dtype.itemsize
    return torch.empty(*shape[:-1], (shape[-1] + per - 1) // per * per, dtype=dtype, device="cuda")[..., :shape[-1]]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 23)


def _logits(g, T, E, masked):
    """Scores of tokens by experts: some experts liked by all, some tokens sure of theirs."""
    s = torch.randn(T, E, generator=g, device="cuda")
    s = s * torch.exp(0.5 * torch.randn(T, 1, generator=g, device="cuda")) + 0.7 * torch.randn(E, generator=g, device="cuda")
    if masked:  # experts that are away, and padded tokens that go to none
        s[:, torch.rand(E, generator=g, device="cuda") < 0.1] = -math.inf
        s[torch.rand(T, generator=g, device="cuda") < 0.02] = -math.inf
    return s


def _group(ids, groups):
    """(slots, rows, offsets) of ids [T, k]: the entries sorted by group, those of no group behind the last."""
    T, k = ids.shape
    flat = ids.reshape(-1).long()
    key = torch.where((flat < 0) | (flat >= groups), groups, flat)
    order = torch.argsort(key, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k, device=ids.device)
    slots = torch.where(key < groups, place, -1).reshape(T, k)
    counts = torch.bincount(key, minlength=groups + 1)[:groups]
    offsets = torch.zeros(groups + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = counts.cumsum(0)
    return slots.to(I32), torch.div(order, k, rounding_mode="floor").to(I32), offsets.to(I32)


def _top(logits, k):
    """The k largest of each row, the lowest index first among equals."""
    return torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :k]


def prepare(case, seed):
    g = _gen(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=F32)

    def matrix(*shape, scale=1.0):
        out = _rows16(*shape, dtype=dt)
        out.copy_(normal(*shape).mul_(scale))
        return out

    s = {"op": op}
    if op in ("route", "route_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = _logits(g, T, E, case["T"] % 2 == 0).to(dt)
        s["k"], s["normalize"] = k, case["normalize"]
        if op == "route_bwd":
            ids = _top(s["logits"].float(), k)
            s["ids"] = torch.where(s["logits"].gather(1, ids) > -math.inf, ids, -1).to(I32)
            s["dweights"] = normal(T, k).mul_(0.01)
        return s
    if op in ("combine", "combine_bwd"):
        T, C, k = case["T"], case["C"], case["k"]
        ids = torch.topk(normal(T, max(8, k)), k, dim=1)[1]
        if op == "combine":  # some answers are missing: experts that were full
            ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < 0.02, -1, ids)
        s["slots"] = _group(ids, max(8, k))[0]
        s["y"] = matrix(T * k, C)
        s["weights"] = torch.softmax(normal(T, k), 1)
        if op == "combine_bwd":
            s["dout"] = matrix(T, C, scale=0.01)
        return s
    if op in ("grouped", "grouped_bwd"):
        T, k, E, K, n = (case[v] for v in ("T", "k", "E", "K", "n"))
        ids = _top(_logits(g, T, E, False), k)
        _, rows, s["offsets"] = _group(ids, E)
        s["rows"] = rows if case["gather"] else None
        s["x"] = matrix(T if case["gather"] else T * k, K)
        s["w"] = _rows16(E, K, n, dtype=dt)
        for e in range(E):
            s["w"][e].copy_(normal(K, n).mul_(1 / math.sqrt(K)))
        if op == "grouped_bwd":
            s["dy"] = matrix(T * k, n, scale=0.02)
        ends = s["offsets"].tolist()  # the plain form's plan
        s["spans"] = [(e, ends[e], ends[e + 1]) for e in range(E) if ends[e + 1] > ends[e]]
        return s
    # requests of about `runs` tokens each, one in sixteen of them without an adapter
    T, K, n, r, R = (case[v] for v in ("T", "K", "n", "r", "R"))
    pick = torch.randint(0, R, (T,), generator=g, device="cuda")
    pick = torch.where(torch.rand(T, generator=g, device="cuda") < 1 / 16, -1, pick)
    starts = torch.rand(T, generator=g, device="cuda") < 1 / case["runs"]
    s["ids"] = pick[starts.long().cumsum(0).clamp_max(T - 1)].to(I32)
    s["x"] = matrix(T, K)
    s["a"] = matrix(R, K, r, scale=1 / math.sqrt(K))
    s["b"] = matrix(R, r, n, scale=1 / math.sqrt(r))
    s["scale"] = torch.exp(0.5 * normal(R))
    if op == "adapter":
        s["base"] = matrix(T, n)
    else:
        s["dy"] = matrix(T, n, scale=0.02)
        s["base"] = matrix(T, K, scale=0.02)
        s["h"] = matrix(T, r)
        s["h"][s["ids"] < 0] = 0
    s["members"] = [(i, (s["ids"] == i).nonzero()[:, 0]) for i in s["ids"].unique().tolist() if i >= 0]  # the plain form's
    return s


# ---- the plain forms -----------------------------------------------------------------------------------------------

def _route(s):
    logits, k = s["logits"].float(), s["k"]
    T, E = logits.shape
    ids = _top(logits, k)
    best = logits.gather(1, ids)
    there = best > -math.inf
    if s["normalize"]:
        e = torch.where(there, torch.exp(best - best[:, :1]), 0.0)
        w = e / e.sum(1, keepdim=True)
    else:
        top = logits.amax(1, keepdim=True)
        w = torch.exp(best - top) / torch.exp(logits - top).sum(1, keepdim=True)
    w = torch.where(there, w, 0.0)
    ids = torch.where(there, ids, -1).to(I32)
    return (w, ids, *_group(ids, E))


def _route_bwd(s):
    logits, ids, g = s["logits"].float(), s["ids"].long(), s["dweights"]
    there, at = ids >= 0, ids.clamp_min(0)
    if s["normalize"]:
        best = torch.where(there, logits.gather(1, at), -math.inf)
        top = best.amax(1, keepdim=True)
        w = torch.where(there, torch.exp(best - top), 0.0)
        w = w / w.sum(1, keepdim=True).clamp_min(1.0)
        d = w * (g - (w * g).sum(1, keepdim=True))
        out = torch.zeros_like(logits)
        out.scatter_add_(1, at, torch.where(there, d, 0.0))
    else:
        top = logits.amax(1, keepdim=True)
        top = torch.where(top > -math.inf, top, 0.0)
        p = torch.exp(logits - top)
        p = p / p.sum(1, keepdim=True).clamp_min(1e-30)
        all_g = torch.zeros_like(logits)
        all_g.scatter_add_(1, at, torch.where(there, g, 0.0))
        out = p * (all_g - (p * all_g).sum(1, keepdim=True))
    return out.to(s["logits"].dtype)


def _combine(s):
    slots, w = s["slots"].long(), s["weights"]
    T, k = slots.shape
    out = torch.zeros(T, s["y"].shape[1], device="cuda")
    for j in range(k):
        there = slots[:, j] >= 0
        wj = torch.where(there, w[:, j], 0.0)
        out += wj[:, None] * s["y"][slots[:, j].clamp_min(0)].float()
    return out.to(s["y"].dtype)


def _combine_bwd(s):
    slots, w, dout = s["slots"].long(), s["weights"], s["dout"].float()
    dy = torch.empty(s["y"].shape, device="cuda", dtype=s["y"].dtype)
    dw = torch.empty_like(w)
    for j in range(slots.shape[1]):
        dy[slots[:, j]] = (w[:, j, None] * dout).to(dy.dtype)
        dw[:, j] = (dout * s["y"][slots[:, j]].float()).sum(1)
    return dy, dw


def _member_rows(s, a, b):
    return (s["x"][s["rows"][a:b].long()] if s["rows"] is not None else s["x"][a:b]).float()


def _grouped(s):
    n = s["w"].shape[2]
    y = torch.empty(s["spans"][-1][2], n, dtype=s["x"].dtype, device="cuda")
    for e, a, b in s["spans"]:
        y[a:b] = _member_rows(s, a, b) @ s["w"][e].float()
    return y


def _grouped_bwd(s):
    E, K, n = s["w"].shape
    dx = torch.empty(s["spans"][-1][2], K, dtype=s["x"].dtype, device="cuda")
    dw = torch.zeros(E, K, n, dtype=s["x"].dtype, device="cuda")
    for e, a, b in s["spans"]:
        g = s["dy"][a:b].float()
        dx[a:b] = g @ s["w"][e].float().T
        dw[e] = _member_rows(s, a, b).T @ g
    return dx, dw


def _adapter(s):
    x, y = s["x"], s["base"].float()
    h = torch.zeros(x.shape[0], s["a"].shape[2], dtype=x.dtype, device="cuda")
    for i, at in s["members"]:
        hi = x[at].float() @ s["a"][i].float()
        h[at] = hi.to(x.dtype)
        y[at] += s["scale"][i] * (hi @ s["b"][i].float())
    return y.to(x.dtype), h


def _adapter_bwd(s):
    x, dx = s["x"], s["base"].float()
    da, db = torch.zeros_like(s["a"]), torch.zeros_like(s["b"])
    for i, at in s["members"]:
        g = s["dy"][at].float()
        dh = s["scale"][i] * (g @ s["b"][i].float().T)
        dx[at] += dh @ s["a"][i].float().T
        da[i] = x[at].float().T @ dh
        db[i] = s["scale"][i] * (s["h"][at].float().T @ g)
    return dx.to(x.dtype), da, db


def run(state):
    s, op = state, state["op"]
    if not own:
        return {"route": _route, "route_bwd": _route_bwd, "combine": _combine, "combine_bwd": _combine_bwd,
                "grouped": _grouped, "grouped_bwd": _grouped_bwd, "adapter": _adapter, "adapter_bwd": _adapter_bwd}[op](s)
    from offload_streamed_gb300 import tiled_linear as tl
    if op == "route":
        return tl.route(s["logits"], s["k"], normalize=s["normalize"])
    if op == "route_bwd":
        return tl.route_backward(s["dweights"], s["logits"], s["ids"], normalize=s["normalize"])
    if op == "combine":
        return tl.combine(s["y"], s["slots"], s["weights"])
    if op == "combine_bwd":
        return tl.combine_backward(s["dout"], s["slots"], s["y"], s["weights"])
    if op == "grouped":
        return tl.grouped_linear(s["x"], s["w"], s["offsets"], s["rows"])
    if op == "grouped_bwd":
        return tl.grouped_linear_backward(s["x"], s["dy"], s["w"], s["offsets"], s["rows"])
    if op == "adapter":
        return tl.adapter_linear(s["x"], s["a"], s["b"], s["ids"], base=s["base"], scale=s["scale"])
    return tl.adapter_linear_backward(s["x"], s["h"], s["dy"], s["a"], s["b"], s["ids"], base=s["base"], scale=s["scale"])


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------

def _exact_route(s):
    l = s["logits"].to(F64)
    T, E = l.shape
    k = s["k"]
    left, ids = l.clone(), []
    for _ in range(k):  # the largest, then the largest of the rest: amax and the first place that holds it
        top = left.amax(1, keepdim=True)
        at = torch.where(left == top, torch.arange(E, device="cuda"), E).amin(1)
        ids.append(torch.where(top[:, 0] > -math.inf, at, -1))
        left.scatter_(1, at[:, None], -math.inf)
    ids = torch.stack(ids, 1)
    v = torch.where(ids >= 0, l.gather(1, ids.clamp_min(0)), -math.inf)
    over = v if s["normalize"] else l
    w = torch.exp(v - torch.logsumexp(over, 1, keepdim=True))
    w = torch.where(ids >= 0, w, 0.0)
    # an entry's place: the entries of lower experts, and the earlier ones of its own
    flat = ids.reshape(-1)
    member = torch.nn.functional.one_hot(torch.where(flat < 0, E, flat), E + 1).to(I32)
    count = member.sum(0)
    ends = count.cumsum(0)
    earlier = (member.cumsum(0) - member).gather(1, torch.where(flat < 0, E, flat)[:, None])[:, 0]
    place = (ends - count)[torch.where(flat < 0, E, flat)] + earlier
    rows = torch.empty(T * k, dtype=I32, device="cuda")
    rows[place] = (torch.arange(T * k, device="cuda") // k).to(I32)
    slots = torch.where(flat < 0, -1, place).reshape(T, k).to(I32)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), ends[:E]]).to(I32)
    return w, ids.to(I32), slots, rows, offsets


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "route":
        return _exact_route(s)
    if op == "route_bwd":
        l = s["logits"].to(F64).requires_grad_(True)
        there = s["ids"] >= 0
        at = torch.where(there, s["ids"], 0).long()
        some = there.any(1)  # the gradient of the chosen weights' sum with dweights, by differentiation
        v = l[some].gather(1, at[some]).masked_fill(~there[some], -math.inf)
        w = torch.softmax(v, 1) if s["normalize"] else torch.exp(v - torch.logsumexp(l[some], 1, keepdim=True))
        torch.where(there[some], w * s["dweights"][some].to(F64), 0.0).sum().backward()
        return l.grad
    if op == "combine":
        at = torch.where(s["slots"] < 0, 0, s["slots"]).long()
        w = torch.where(s["slots"] < 0, 0.0, s["weights"].to(F64))
        out = torch.zeros(at.shape[0], s["y"].shape[1], dtype=F64, device="cuda")
        for j in range(at.shape[1]):
            out.addcmul_(w[:, j, None], s["y"].index_select(0, at[:, j]).to(F64))
        return out
    if op == "combine_bwd":
        T, k = s["slots"].shape
        flat = s["slots"].reshape(-1).long()
        token = torch.empty_like(flat)
        token[flat] = torch.arange(T * k, device="cuda") // k  # the token of each place
        share = torch.empty(T * k, dtype=F64, device="cuda")
        share[flat] = s["weights"].reshape(-1).to(F64)
        d = s["dout"].to(F64)[token]
        dot = torch.einsum("rc,rc->r", d, s["y"].to(F64))
        return d * share[:, None], dot[flat].reshape(T, k)
    if op in ("grouped", "grouped_bwd"):
        off = s["offsets"].cpu().numpy()
        E, K, n = s["w"].shape
        x = s["x"].to(F64)
        x = x if s["rows"] is None else x.index_select(0, s["rows"][:int(off[E])].long())
        parts = [(e, slice(int(off[e]), int(off[e + 1]))) for e in range(E)]
        if op == "grouped":
            return torch.cat([torch.einsum("tk,kn->tn", x[p], s["w"][e].to(F64)) for e, p in parts])
        dy = s["dy"].to(F64)
        dx = torch.cat([torch.einsum("tn,kn->tk", dy[p], s["w"][e].to(F64)) for e, p in parts])
        return dx, torch.stack([torch.einsum("tk,tn->kn", x[p], dy[p]) for _, p in parts])
    # each adapter over all rows, the others' scaled by nought
    x, a, b, base = (s[v].to(F64) for v in ("x", "a", "b", "base"))
    owns = [((s["ids"] == i).nonzero()[:, 0], s["scale"][i].to(F64)) for i in range(a.shape[0])]
    if op == "adapter":
        y, h = base.clone(), torch.zeros(x.shape[0], a.shape[2], dtype=F64, device="cuda")
        for i, (at, f) in enumerate(owns):
            h.index_add_(0, at, x[at] @ a[i])
            y.index_add_(0, at, f * (h[at] @ b[i]))
        return y, h
    dy, h, dx = s["dy"].to(F64), s["h"].to(F64), base.clone()
    da, db = torch.zeros_like(a), torch.zeros_like(b)
    for i, (at, f) in enumerate(owns):
        dh = f * torch.einsum("tn,rn->tr", dy[at], b[i])
        dx.index_add_(0, at, torch.einsum("tr,kr->tk", dh, a[i]))
        da[i], db[i] = torch.einsum("tk,tr->kr", x[at], dh), f * torch.einsum("tr,tn->rn", h[at], dy[at])
    return dx, da, db
