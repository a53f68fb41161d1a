"""The operators whose weight depends on the row in 64 bits, from their definitions, with the error that each kernel may
make, element by element.

Roundings counted: a result's own, `half(dtype)` of its value (half a step: finfo.eps / 2, and below the smallest normal
number half the smallest step); in a sum of n products in 32 bits, one of 2^-23 of the sum of magnitudes for each (the
tensor cores' additions may cut off, which is twice a rounding)."""
import torch

STEP = 2.0 ** -23


def half(dtype):
    return torch.finfo(dtype).eps / 2


def floor_of(dtype):
    """Half a step among the subnormal numbers."""
    f = torch.finfo(dtype)
    return f.tiny * f.eps / 2


def rounded(ref, before, dtype):
    """Bound for a value that is off by `before` and then rounded to dtype."""
    return half(dtype) * (ref.abs() + before) + before + floor_of(dtype)


def check(name, got, ref, bound):
    got = got.double()
    assert got.shape == ref.shape, f"{name}: {tuple(got.shape)} for {tuple(ref.shape)}"
    bad = ~((got - ref).abs() <= bound)
    if bad.any():
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, first at {at}: {got[at].item()} for {ref[at].item()}, "
                             f"allowed {bound[at].item() if bound.shape == ref.shape else bound}")


def group(ids, groups):
    """slots, rows, offsets of ids [T, k] by counting, entry by entry."""
    T, k = ids.shape
    flat = [i if 0 <= i < groups else groups for i in ids.reshape(-1).tolist()]
    counts, begin, total = [0] * (groups + 1), [], 0
    for i in flat:
        counts[i] += 1
    for c in counts:
        begin.append(total)
        total += c
    at, slots, rows = list(begin), [], [0] * (T * k)
    for e, i in enumerate(flat):
        rows[at[i]] = e // k
        slots.append(at[i] if i < groups else -1)
        at[i] += 1
    return (torch.tensor(slots, dtype=torch.int32).reshape(T, k), torch.tensor(rows, dtype=torch.int32),
            torch.tensor(begin, dtype=torch.int32))


def spans(offsets):
    o = offsets.tolist()
    return [(g, o[g], o[g + 1]) for g in range(len(o) - 1)]


def grouped(x, w, offsets, rows=None):
    """(y, bound)"""
    K, n = w.shape[1:]
    x64 = x.double() if rows is None else x.double()[rows.long()]
    y, mag = (torch.zeros(x64.shape[0], n, dtype=torch.float64, device=x.device) for _ in range(2))
    for g, a, b in spans(offsets):
        y[a:b] = x64[a:b] @ w[g].double()
        mag[a:b] = x64[a:b].abs() @ w[g].double().abs()
    return y, rounded(y, K * STEP * mag, x.dtype)


def grouped_backward(x, dy, w, offsets, rows=None):
    """(dx, bound), (dw, bound)"""
    E, K, n = w.shape
    x64, g64 = (x.double() if rows is None else x.double()[rows.long()]), dy.double()
    dx, mx = (torch.zeros(dy.shape[0], K, dtype=torch.float64, device=x.device) for _ in range(2))
    dw, mw = (torch.zeros(E, K, n, dtype=torch.float64, device=x.device) for _ in range(2))
    for g, a, b in spans(offsets):
        dx[a:b], mx[a:b] = g64[a:b] @ w[g].double().T, g64[a:b].abs() @ w[g].double().abs().T
        dw[g], mw[g] = x64[a:b].T @ g64[a:b], (b - a) * (x64[a:b].abs().T @ g64[a:b].abs())
    return (dx, rounded(dx, n * STEP * mx, x.dtype)), (dw, rounded(dw, STEP * mw, x.dtype))


def between(ref, before, dtype):
    """What an intermediate result is off by when it is handed on in two parts of dtype."""
    return before + half(dtype) ** 2 * (ref.abs() + before) + floor_of(dtype)


def members(ids, adapters):
    return [(i, (ids == i).nonzero()[:, 0]) for i in range(adapters)]


def adapter(x, a, b, ids, base, scale):
    """(y, bound), (h, bound)"""
    T, K, n, r, dt = x.shape[0], x.shape[1], b.shape[2], a.shape[2], x.dtype
    z = lambda *s: torch.zeros(*s, dtype=torch.float64, device=x.device)  # noqa: E731
    h, eh, y, ey = z(T, r), z(T, r), z(T, n), z(T, n)
    if base is not None:
        y += base.double()
        ey += 2 * STEP * y.abs()
    for i, at in members(ids, a.shape[0]):
        s, x64, a64, b64 = abs(float(scale[i])), x[at].double(), a[i].double(), b[i].double()
        h[at], eh[at] = x64 @ a64, K * STEP * (x64.abs() @ a64.abs())
        off = between(h[at], eh[at], dt)
        y[at] += float(scale[i]) * (h[at] @ b64)
        ey[at] += s * (off @ b64.abs() + (2 * r + 3) * STEP * ((h[at].abs() + off) @ b64.abs()))
    return (y, rounded(y, ey, dt)), (h, rounded(h, eh, dt))


def adapter_backward(x, h, dy, a, b, ids, base, scale):
    """(dx, bound), (da, bound), (db, bound)"""
    T, K, n, r, dt = x.shape[0], x.shape[1], b.shape[2], a.shape[2], x.dtype
    z = lambda *s: torch.zeros(*s, dtype=torch.float64, device=x.device)  # noqa: E731
    dx, ex, da, ea, db, eb = z(T, K), z(T, K), z(*a.shape), z(*a.shape), z(*b.shape), z(*b.shape)
    if base is not None:
        dx += base.double()
        ex += 2 * STEP * dx.abs()
    for i, at in members(ids, a.shape[0]):
        s, x64, g, a64, b64, h64 = float(scale[i]), x[at].double(), dy[at].double(), a[i].double(), b[i].double(), h[at].double()
        dh = s * (g @ b64.T)
        off = between(dh, (n + 2) * STEP * abs(s) * (g.abs() @ b64.abs().T), dt)
        dx[at] += dh @ a64.T
        ex[at] += off @ a64.abs().T + (2 * r + 3) * STEP * ((dh.abs() + off) @ a64.abs().T)
        da[i] = x64.T @ dh
        ea[i] = x64.abs().T @ off + (2 * len(at) + 8) * STEP * (x64.abs().T @ (dh.abs() + off))
        db[i] = s * (h64.T @ g)
        eb[i] = abs(s) * (len(at) + 8) * STEP * (h64.abs().T @ g.abs())
    return (dx, rounded(dx, ex, dt)), (da, rounded(da, ea, dt)), (db, rounded(db, eb, dt))
