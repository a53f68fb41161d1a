"""The router: the choice of experts and the entries' order exactly, weights, sums and gradients against 64 bits.

Bounds: a weight is a quotient of exponentials in 32 bits: 2^-24 of the exponent's argument, two steps for each
exponential and one for each addition; the gradient's subtraction adds those of both sides.  A combined row is k
multiply-adds in 32 bits, rounded once; a weight's gradient sums `cols` products in 32 bits."""
import pytest
import torch

from rows_reference import STEP, check, floor_of, group, half, rounded

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def tl():
    import __graft_entry__ as g
    g.build()
    from offload_streamed_gb300 import tiled_linear
    yield tiled_linear
    tiled_linear.check_operators()


def scores(T, E, dtype, seed, masked=True):
    g = torch.Generator().manual_seed(seed)
    s = torch.randn(T, E, generator=g) * 2
    if dtype == F32:  # equal scores occur in 32 bits, too
        s = (s * 4).round() / 4
    if masked:
        s[torch.rand(T, E, generator=g) < 0.1] = -float("inf")
        s[torch.rand(T, E, generator=g) < 0.02] = float("nan")
        s[torch.rand(T, generator=g) < 0.1] = -float("inf")
    s[torch.rand(T, E, generator=g) < 0.05] = 0.0
    s[torch.rand(T, E, generator=g) < 0.05] = -0.0
    return s.to(dtype)


def choice(logits, k, normalize):
    """ids and weights, a round for each rank, in 64 bits on the host."""
    l = torch.where(logits.isnan(), -float("inf"), logits.double())
    T, E = l.shape
    left, ids = l.clone(), torch.full((T, k), -1)
    for j in range(k):
        best = left.max(1).values
        first = (left == best[:, None]).float().argmax(1)  # the first that holds it
        ids[:, j] = torch.where(best > -float("inf"), first, -1)
        left[torch.arange(T), first] = -float("inf")
    there = ids >= 0
    v = torch.where(there, l.gather(1, ids.clamp_min(0)), -float("inf"))
    over = v if normalize else l
    w = torch.where(there, torch.exp(v - torch.logsumexp(over, 1, keepdim=True)), 0.0)
    return ids.int(), w


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 7, 7), (32, 128, 4), (128, 33, 8), (129, 64, 2), (1000, 256, 8), (40, 300, 32),
                                   (700, 1024, 3), (5003, 40, 6)])
def test_route(tl, T, E, k, normalize, dtype):
    logits = scores(T, E, dtype, T + E)
    got = tl.route(logits.cuda(), k, normalize=normalize)
    ids, w = choice(logits, k, normalize)
    assert torch.equal(got[1].cpu(), ids)
    assert torch.equal(got[0].cpu() == 0, w == 0)
    check("weights", got[0].cpu(), w, w * (40 + E) * STEP + 1e-37)
    for a, b in zip(got[2:], group(ids, E)):
        assert torch.equal(a.cpu(), b)


def test_route_takes_strides_and_no_tokens(tl):
    logits = scores(50, 40, F32, 1).cuda()
    wide = torch.empty(50, 57, device="cuda")
    wide[:, 3:43] = logits
    for a, b in zip(tl.route(wide[:, 3:43], 5), tl.route(logits, 5)):
        assert torch.equal(a, b)
    w, ids, slots, rows, offsets = tl.route(logits[:0], 5)
    assert w.shape == (0, 5) and rows.shape == (0,) and offsets.tolist() == [0] * 41


@pytest.mark.parametrize("T,k,groups", [(1, 1, 1), (17, 3, 5), (8192, 1, 64), (8193, 1, 3), (3000, 4, 1024), (200000, 2, 37), (700000, 2, 9)])
def test_group_rows(tl, T, k, groups):
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(-2, groups + 2, (T, k), generator=g, dtype=torch.int32)
    for a, b in zip(tl.group_rows(ids.cuda(), groups), group(ids, groups)):
        assert torch.equal(a.cpu(), b)
    same = torch.full((T, k), groups - 1, dtype=torch.int32)  # all in one group
    for a, b in zip(tl.group_rows(same.cuda(), groups), group(same, groups)):
        assert torch.equal(a.cpu(), b)


def gradient(l, ids, dw, normalize):
    """dlogits in 64 bits and the magnitude that its subtraction works on."""
    l, g = torch.where(l.isnan(), -float("inf"), l.double()), dw.double()
    there, at = ids >= 0, ids.clamp_min(0).long()
    full = torch.zeros_like(l).scatter_add_(1, at, torch.where(there, g, 0.0))
    big = torch.zeros_like(l).scatter_add_(1, at, torch.where(there, g.abs(), 0.0))
    p = l
    if normalize:
        p = torch.full_like(l, -float("inf"))
        for j in range(ids.shape[1]):
            rows = there[:, j].nonzero()[:, 0]
            p[rows, at[rows, j]] = l[rows, at[rows, j]]
    p = torch.nan_to_num(torch.softmax(p, 1), nan=0.0)
    return p * (full - (p * full).sum(1, keepdim=True)), p * (big + (p * big).sum(1, keepdim=True))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (33, 7, 7), (300, 64, 2), (50, 1024, 8), (9, 100, 32)])
def test_route_backward(tl, T, E, k, normalize, dtype):
    logits = scores(T, E, dtype, T)
    ids, _ = choice(logits, k, normalize)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(1))
    got = tl.route_backward(dw.cuda(), logits.cuda(), ids.cuda(), normalize=normalize)
    ref, size = gradient(logits, ids, dw, normalize)
    check("dlogits", got.cpu(), ref, rounded(ref, (60 + E) * STEP * size, dtype) + 1e-37)


def test_route_gradient_by_differences(tl):
    """The weights' change along a direction, in 64 bits, against the gradient's."""
    T, E, k = 40, 24, 3
    logits = scores(T, E, F32, 5, masked=False)
    g = torch.Generator().manual_seed(2)
    dw, step = torch.randn(T, k, generator=g), torch.randn(T, E, generator=g).double()
    for normalize in (True, False):
        ids, _ = choice(logits, k, normalize)
        out = tl.route_backward(dw.cuda(), logits.cuda(), ids.cuda(), normalize=normalize).cpu().double()
        at = ids.long()

        def total(eps):
            l = logits.double() + eps * step
            v = l.gather(1, at)
            return (torch.exp(v - torch.logsumexp(v if normalize else l, 1, keepdim=True)) * dw).sum()

        e = 1e-5  # truncation e^2, cancellation 2^-52 / e: both far below
        slope = (total(e) - total(-e)) / (2 * e)
        # 32-bit gradient: its error, at most 100 steps of each element, times the direction
        assert abs((out * step).sum() - slope) <= 100 * STEP * (out * step).abs().sum() + 1e-7


def placed(T, k, rows, dropped, seed):
    g = torch.Generator().manual_seed(seed)
    slots = torch.randperm(rows, generator=g)[:T * k].reshape(T, k).int()
    slots[torch.rand(T, k, generator=g) < dropped] = -1
    return slots


def matrix(rows, cols, dtype, seed, gap=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    wide = torch.randn(rows, cols + gap, generator=g, device="cuda").to(dtype)
    return wide[:, :cols]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("gap", [0, 8, 3])
@pytest.mark.parametrize("T,k,cols", [(1, 1, 1), (1, 2, 16), (37, 8, 1000), (300, 2, 264), (5, 32, 4099), (3, 5, 20000)])
def test_combine_and_backward(tl, T, k, cols, gap, dtype):
    rows = T * k + 3
    slots, y = placed(T, k, rows, 0.2, T), matrix(rows, cols, dtype, 1, gap)
    w = torch.randn(T, k, generator=torch.Generator().manual_seed(3))
    if k > 1:  # a missing answer's weight does not matter
        slots[0, 0], w[0, 0] = -1, float("nan")
    used = set(slots[slots >= 0].tolist())
    for i, v in zip([i for i in range(rows) if i not in used], (float("nan"), float("inf"))):
        y[i] = v  # nor does a row that nobody names
    there = slots >= 0
    w64 = torch.where(there, w.double(), 0.0).cuda()
    picked = torch.where(there.cuda()[..., None], y.double()[slots.clamp_min(0).long().cuda()], 0.0)  # [T, k, cols]
    for weights, f in ((w.cuda(), w64), (None, there.double().cuda())):
        out = tl.combine(y, slots.cuda(), weights)
        ref, mag = torch.einsum("tk,tkc->tc", f, picked), torch.einsum("tk,tkc->tc", f.abs(), picked.abs())
        check("out", out, ref, rounded(ref, k * STEP * mag, dtype))
        dout = matrix(T, cols, dtype, 2, gap)
        dy, dw = tl.combine_backward(dout, slots.cuda(), y, weights)
        ref = f[..., None] * dout.double()[:, None]
        at = there.cuda()
        check("dy", dy[slots.cuda()[at].long()], ref[at], rounded(ref[at], 0.0, dtype))
        ref, mag = (picked * dout.double()[:, None]).sum(2), (picked * dout.double()[:, None]).abs().sum(2)
        check("dweights", dw, ref, cols * STEP * mag)
    dy, none = tl.combine_backward(dout, slots.cuda(), weights=w.cuda())  # without y: as many rows as entries
    assert none is None and dy.shape == (T * k, cols)


def test_rows_that_nobody_names_keep_their_bits(tl):
    T, k, cols, rows = 20, 2, 136, 50
    slots, dout = placed(T, k, rows, 0.3, 1).cuda(), matrix(T, cols, BF16, 2)
    dy = torch.full((rows, cols), 7.0, dtype=BF16, device="cuda")
    tl.tiled_linear_combine_backward(T, k, cols, rows, 0, dout.data_ptr(), cols, slots.data_ptr(), None, 0, None, dy.data_ptr(), cols, None,
                                     torch.cuda.current_stream().cuda_stream)
    left = torch.ones(rows, dtype=torch.bool)
    left[slots[slots >= 0].long().cpu()] = False
    assert left.any() and (dy[left.cuda()] == 7).all()


def test_slots_outside_add_nothing(tl):
    y, big = matrix(6, 32, F32, 1), torch.tensor([[0, 6], [-5, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    out = tl.combine(y, big)
    assert torch.equal(out[0], y[0]) and (out[1] == 0).all()
    dy, dw = tl.combine_backward(matrix(2, 32, F32, 2), big, y)
    assert (dw.reshape(-1)[1:] == 0).all() and dy.shape == y.shape


def test_no_tokens(tl):
    y, none = matrix(4, 16, BF16, 1), torch.empty(0, 2, dtype=torch.int32, device="cuda")
    assert tl.combine(y, none).shape == (0, 16)
    dy, dw = tl.combine_backward(y[:0], none, y)
    assert dy.shape == (4, 16) and dw.shape == (0, 2)


def test_gathered_rows_and_their_gradient(tl):
    """x[rows] and the sum over a token's places are each other's adjoint."""
    T, E, k, cols = 200, 16, 3, 72
    _, _, slots, rows, _ = tl.route(scores(T, E, F32, 3, masked=False).cuda(), k)
    x, g = matrix(T, cols, F32, 4), matrix(T * k, cols, F32, 5)
    back = tl.combine(g, slots)
    lhs, rhs = (x[rows.long()].double() * g.double()).sum(), (x.double() * back.double()).sum()
    assert abs(lhs - rhs) <= (k + 1) * STEP * (x[rows.long()].double() * g.double()).abs().sum()


def test_half_a_step():  # the bounds' own unit
    assert half(BF16) == 2.0 ** -8 and half(F16) == 2.0 ** -11 and floor_of(F16) == 2.0 ** -25
