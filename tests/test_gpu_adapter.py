"""Low-rank adapters (through the package's functions, so through the C ABI) against 64 bits, element by element; the
bounds are those of rows_reference.py."""
import pytest
import torch

from rows_reference import adapter, adapter_backward, check

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def tl():
    import __graft_entry__ as g
    g.build()
    from offload_streamed_gb300 import tiled_linear
    yield tiled_linear
    tiled_linear.check_operators()


def normal(seed, *shape, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def owners(seed, T, R, runs):
    """ids of runs of about `runs` rows, some of no adapter."""
    g = torch.Generator().manual_seed(seed)
    pick = torch.randint(-1, R + 1, (T,), generator=g, dtype=torch.int32)
    return pick[(torch.rand(T, generator=g) < 1 / runs).long().cumsum(0).clamp_max(T - 1)].cuda()


def case(T, K, n, r, R, dtype, runs=3, seed=0):
    x, a, b = normal(seed + 1, T, K, dtype=dtype), normal(seed + 2, R, K, r, dtype=dtype), normal(seed + 3, R, r, n, dtype=dtype)
    return x, a / K ** 0.5, b / r ** 0.5, owners(seed, T, R, runs), torch.exp(normal(seed + 4, R, dtype=F32))


def both(tl, x, a, b, ids, scale, base_dtype=None, seed=0):
    T, K, n, r = x.shape[0], x.shape[1], b.shape[2], a.shape[2]
    base = base_dx = None
    if base_dtype is not None:
        base, base_dx = normal(seed + 5, T, n, dtype=base_dtype), normal(seed + 6, T, K, dtype=base_dtype)
    scales = scale if torch.is_tensor(scale) else [scale] * a.shape[0]
    y, h = tl.adapter_linear(x, a, b, ids, base=base, scale=scale)
    for name, got, ref in zip(("y", "h"), (y, h), adapter(x, a, b, ids, base, scales)):
        check(name, got, *ref)
    dy = normal(seed + 7, T, n, dtype=x.dtype)
    got = tl.adapter_linear_backward(x, h, dy, a, b, ids, base=base_dx, scale=scale)
    for name, g, ref in zip(("dx", "da", "db"), got, adapter_backward(x, h, dy, a, b, ids, base_dx, scales)):
        check(name, g, *ref)
    tl.check_operators()


@pytest.mark.parametrize("base", [None, BF16, F32])
@pytest.mark.parametrize("r", [1, 4, 8, 16, 24, 32, 64, 100, 128])
@pytest.mark.parametrize("T", [1, 20, 64, 65, 300])
def test_ranks(tl, T, r, base):
    both(tl, *case(T, 264, 392, r, 5, BF16), base_dtype=base)


@pytest.mark.parametrize("T,K,n,R,runs", [(3, 1, 1, 1, 1), (70, 7, 300, 3, 2), (130, 300, 7, 2, 50), (33, 65, 129, 40, 1),
                                          (1000, 513, 1030, 3, 300), (2000, 72, 64, 900, 2), (3000, 72, 136, 1024, 3), (64, 4099, 2056, 64, 1)])
def test_odd_sizes(tl, T, K, n, R, runs):
    both(tl, *case(T, K, n, 16, R, F16, runs), base_dtype=F16)


@pytest.mark.parametrize("T,K,n,r,R,runs", [(32, 8192, 4096, 16, 64, 1), (1, 8192, 512, 64, 1, 1), (2048, 4096, 1024, 32, 4, 400), (3000, 256, 4096, 64, 1, 3000)])
def test_long_reductions(tl, T, K, n, r, R, runs):
    x, a, b, ids, scale = case(T, K, n, r, R, BF16, runs)
    both(tl, x, a, b, ids, 0.25, base_dtype=BF16)


def test_rows_without_an_adapter(tl):
    """y is base and h zero, bit for bit; with no adapter at all the gradients are zeros."""
    for T in (7, 200):
        x, a, b, ids, scale = case(T, 128, 264, 16, 3, BF16)
        base, dy = normal(9, T, 264), normal(10, T, 264)
        ids[::2], ids[1] = -1, 0
        y, h = tl.adapter_linear(x, a, b, ids, base=base, scale=scale)
        assert torch.equal(y[::2], base[::2]) and not h[::2].any() and h[1].any()
        none = torch.full_like(ids, 3)
        x.fill_(float("inf"))
        dx, da, db = tl.adapter_linear_backward(x, h, dy, a, b, none, base=x, scale=scale)
        assert torch.equal(dx, x) and not da.any() and not db.any()
        y, h = tl.adapter_linear(x, a, b, none)
        assert not y.any() and not h.any()


def test_other_rows_and_adapters_do_not_matter(tl):
    """Infinities and NaN in one request's rows or one adapter's weights stay with it."""
    for T in (40, 300):
        x, a, b, ids, scale = case(T, 200, 264, 16, 4, BF16)
        h0, dy = normal(8, T, 16), normal(9, T, 264)
        good = *tl.adapter_linear(x, a, b, ids, scale=scale), *tl.adapter_linear_backward(x, h0, dy, a, b, ids, scale=scale)
        bad_rows = ids == 1
        assert bad_rows.any() and not bad_rows.all()
        x[bad_rows], dy[bad_rows], h0[bad_rows] = float("inf"), float("nan"), float("nan")
        x[ids < 0], dy[ids < 0] = float("nan"), float("nan")
        a[1], b[1] = float("nan"), float("inf")
        bad = *tl.adapter_linear(x, a, b, ids, scale=scale), *tl.adapter_linear_backward(x, h0, dy, a, b, ids, scale=scale)
        keep = ~bad_rows
        for i in (0, 1, 2):
            assert torch.equal(good[i][keep], bad[i][keep]), i
        for i in (3, 4):
            for e in (0, 2, 3):
                assert torch.equal(good[i][e], bad[i][e]), (i, e)


def test_strided_operands(tl):
    for at in (0, 8, 3):
        T, K, n, r, R = 150, 136, 200, 16, 3
        x = normal(1, T, K + 24)[:, at:at + K]
        a, b = normal(2, R, K + 3, r + 24)[:, 1:1 + K, at:at + r], normal(3, R, r + 3, n + 24)[:, 2:2 + r, at:at + n]
        base = normal(5, T, n + 24)[:, at:at + n]
        ids = owners(1, T, R, 4)
        for rows in (T, 30):
            y, h = tl.adapter_linear(x[:rows], a, b, ids[:rows], base=base[:rows])
            for name, g, ref in zip(("y", "h"), (y, h), adapter(x[:rows], a, b, ids[:rows], base[:rows], [1.0] * R)):
                check(name, g, *ref)


def test_into_base(tl):
    """y may be base (through the C ABI): the shared projection's result gains the adapters'."""
    for T in (10, 300):
        K, n, r, R = 256, 520, 16, 3
        x, a, b, ids, scale = case(T, K, n, r, R, BF16)
        y = normal(6, T, n)
        want, _ = tl.adapter_linear(x, a, b, ids, base=y, scale=scale)
        h = torch.empty(T, r, dtype=BF16, device="cuda")
        need = tl.tiled_linear_adapter_workspace_bytes(T, r, R)
        work = torch.empty(need, dtype=torch.uint8, device="cuda")
        tl.tiled_linear_adapter_forward(T, K, n, r, R, 0, x.data_ptr(), K, a.data_ptr(), r, K * r, b.data_ptr(), n, r * n, ids.data_ptr(),
                                        scale.data_ptr(), 1.0, 0, y.data_ptr(), n, y.data_ptr(), n, h.data_ptr(), r, work.data_ptr(), need,
                                        tl.tiled_linear_operator_error_word(), torch.cuda.current_stream().cuda_stream)
        assert torch.equal(y, want)


def test_no_rows(tl):
    x, a, b, ids, scale = case(1, 64, 72, 8, 2, BF16)
    y, h = tl.adapter_linear(x[:0], a, b, ids[:0])
    assert y.shape == (0, 72) and h.shape == (0, 8)
    dx, da, db = tl.adapter_linear_backward(x[:0], h, y, a, b, ids[:0])
    assert dx.shape == (0, 64) and not da.any() and not db.any()


def test_gradients_by_differences(tl):
    """The layer's change along a direction of x, a and b, in 64 bits: a cubic in the step, whose first derivative the
    differences at one and two give exactly."""
    T, K, n, r, R = 100, 96, 136, 16, 3
    x, a, b, ids, scale = case(T, K, n, r, R, BF16)
    g = normal(8, T, n)
    _, h = tl.adapter_linear(x, a, b, ids, scale=scale)
    vx, va, vb = normal(9, T, K).double(), normal(10, R, K, r).double(), normal(11, R, r, n).double()
    got = tl.adapter_linear_backward(x, h, g, a, b, ids, scale=scale)
    bounds = [e for _, e in adapter_backward(x, h, g, a, b, ids, None, scale)]

    def total(e):
        y = 0.0
        for i in range(R):
            at = (ids == i).nonzero()[:, 0]
            hi = (x[at].double() + e * vx[at]) @ (a[i].double() + e * va[i])
            y = y + float(scale[i]) * ((hi @ (b[i].double() + e * vb[i])) * g[at].double()).sum()
        return y

    slope = (8 * (total(1.0) - total(-1.0)) - (total(2.0) - total(-2.0))) / 12
    said = sum((d.double() * v).sum() for d, v in zip(got, (vx, va, vb)))
    allowed = sum((e * v.abs()).sum() for e, v in zip(bounds, (vx, va, vb)))
    # h came rounded: db is off by that, too
    step = sum(abs(float(scale[i])) * 2.0 ** -8 * ((h[ids == i].double().abs().T @ g[ids == i].double().abs()) * vb[i].abs()).sum() for i in range(R))
    assert abs(said - slope) <= allowed + step


@pytest.mark.parametrize("T", [24, 500])
def test_same_bits_again_and_together(tl, T):
    """Calls on two streams at once, and a captured one replayed with other inputs: the bits of calls alone."""
    K, n, r, R = 512, 640, 16, 4
    x, dy = [normal(s, T, K) for s in range(3)], [normal(s + 3, T, n) for s in range(3)]
    ids = [owners(s, T, R, 5) for s in range(3)]
    _, a, b, _, scale = case(1, K, n, r, R, BF16)

    def call(v, i, g):
        y, h = tl.adapter_linear(v, a, b, i, base=g, scale=scale)
        return y, h, *tl.adapter_linear_backward(v, h, g, a, b, i, base=v, scale=scale)

    want = [call(*c) for c in zip(x, ids, dy)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(20):
        with torch.cuda.stream(streams[i % 2]):
            got.append(call(x[i % 3], ids[i % 3], dy[i % 3]))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(p, q) for p, q in zip(g, want[i % 3])), i
    held = [t.clone() for t in (x[0], ids[0], dy[0])]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(*held)
    for i in range(3):
        for t, s in zip(held, (x[i], ids[i], dy[i])):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want[i])), i
