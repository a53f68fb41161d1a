"""Products grouped by expert (through the package's functions, so through the C ABI) against 64 bits, element by element;
the bounds are those of rows_reference.py."""
import pytest
import torch

from rows_reference import check, grouped, grouped_backward

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


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


def offsets_of(counts):
    return torch.tensor([0, *torch.tensor(counts).cumsum(0).tolist()], dtype=torch.int32, device="cuda")


def indices(seed, R, tokens):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, tokens, (R,), generator=g, dtype=torch.int32).cuda()


# groups of no rows, one, parts of tiles, whole tiles, several; one group; many
COUNTS = {"few": [3, 0, 1, 16, 17], "one": [1], "mixed": [0, 5, 256, 300, 0, 1, 129], "last empty": [70, 200, 0], "large": [700],
          "many": [i % 7 for i in range(200)]}


def both(tl, counts, K, n, dtype, gather, seed=0):
    R = sum(counts)
    off = offsets_of(counts)
    rows = indices(seed, R, 40) if gather else None
    x = normal(seed + 1, 40 if gather else R, K, dtype=dtype)
    w, dy = normal(seed + 2, len(counts), K, n, dtype=dtype), normal(seed + 3, R, n, dtype=dtype)
    check("y", tl.grouped_linear(x, w, off, rows), *grouped(x, w, off, rows))
    got = tl.grouped_linear_backward(x, dy, w, off, rows)
    for name, a, ref in zip(("dx", "dw"), got, grouped_backward(x, dy, w, off, rows)):
        check(name, a, *ref)
    tl.check_operators()


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("K,n", [(64, 64), (128, 256), (200, 136), (1000, 520)])
@pytest.mark.parametrize("counts", COUNTS)
def test_grouped(tl, counts, K, n, gather):
    both(tl, COUNTS[counts], K, n, BF16, gather)


@pytest.mark.parametrize("K,n", [(1, 1), (7, 300), (300, 7), (65, 129), (513, 1030)])
@pytest.mark.parametrize("counts", ["few", "mixed"])
def test_odd_sizes(tl, counts, K, n):
    """Rows that are not whole 16-byte vectors: copied into ones that are, results with gaps."""
    both(tl, COUNTS[counts], K, n, F16, True)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("counts,K,n", [([1, 2, 0, 3], 8192, 512), ([40, 60], 4096, 384), ([1000, 0, 24, 1100], 512, 768), ([1500], 2048, 100)])
def test_long_reductions(tl, counts, K, n, dtype):
    both(tl, counts, K, n, dtype, True)


def test_strided_operands(tl):
    """Columns of wider matrices, on 16-byte boundaries and off them."""
    counts, K, n = [30, 0, 90, 200], 136, 200
    R, off = sum(counts), offsets_of(counts)
    for at in (0, 8, 3):
        x, dy = normal(1, R, K + 24)[:, at:at + K], normal(2, R, n + 24)[:, at:at + n]
        w = normal(3, 4, K + 5, n + 24)[:, 2:2 + K, at:at + n]
        check("y", tl.grouped_linear(x, w, off), *grouped(x, w, off))
        for name, a, ref in zip(("dx", "dw"), tl.grouped_linear_backward(x, dy, w, off), grouped_backward(x, dy, w, off)):
            check(name, a, *ref)


@pytest.mark.parametrize("counts", [[70, 58, 0, 300], [3, 2, 0, 9]])
def test_other_groups_rows_do_not_matter(tl, counts):
    """Infinities and NaN in a group's rows, and behind the last group's, reach no other group."""
    K, n, E = 200, 264, len(counts)
    off = offsets_of(counts)
    R, extra = sum(counts), 40
    x, dy, w = normal(1, R + extra, K), normal(2, R + extra, n), normal(3, E, K, n)
    good = tl.grouped_linear(x, w, off)[:R], *tl.grouped_linear_backward(x, dy, w, off)
    a, b = off[1].item(), off[2].item()
    x[a:b], dy[a:b] = float("inf"), float("nan")
    x[R:], dy[R:], w[2] = float("nan"), float("inf"), float("nan")
    bad = tl.grouped_linear(x, w, off)[:R], *tl.grouped_linear_backward(x, dy, w, off)
    keep = torch.ones(R, dtype=torch.bool, device="cuda")
    keep[a:b] = False
    assert torch.equal(good[0][keep], bad[0][keep]) and torch.equal(good[1][:R][keep], bad[1][:R][keep])
    for e in (0, 2, 3):
        assert torch.equal(good[2][e], bad[2][e])
    assert not torch.isfinite(bad[0][a:b]).any()


def test_rows_of_no_group_keep_their_bits(tl):
    for counts in ([10, 20], [100, 300]):
        R, K, n, extra = sum(counts), 128, 384, 37
        off, x, w = offsets_of(counts), normal(1, R + extra, K), normal(2, 2, K, n)
        y, dx = torch.full((R + extra, n), 7.0, dtype=BF16, device="cuda"), torch.full((R + extra, K), 7.0, dtype=BF16, device="cuda")
        dy, s, err = normal(3, R + extra, n), torch.cuda.current_stream().cuda_stream, tl.tiled_linear_operator_error_word()
        tl.tiled_linear_grouped_forward(R + extra, K, n, 2, 0, x.data_ptr(), K, R + extra, None, w.data_ptr(), n, K * n, off.data_ptr(), y.data_ptr(), n, None, 0, err, s)
        tl.tiled_linear_grouped_dx(R + extra, K, n, 2, 0, dy.data_ptr(), n, w.data_ptr(), n, K * n, off.data_ptr(), dx.data_ptr(), K, err, s)
        assert (y[R:] == 7).all() and (dx[R:] == 7).all()
        check("y", y[:R], *grouped(x[:R], w, off))


def test_results_between_others(tl):
    """Results in columns of wider matrices: what lies beside them keeps its bits."""
    counts = [100, 0, 350, 3]
    R, K, n, E = sum(counts), 136, 264, 4
    off, x, w, dy = offsets_of(counts), normal(1, R, K), normal(2, E, K, n), normal(3, R, n)
    s, err = torch.cuda.current_stream().cuda_stream, tl.tiled_linear_operator_error_word()
    y = torch.full((R, n + 16), 7.0, dtype=BF16, device="cuda")
    dw = torch.full((E, K + 1, n + 8), 7.0, dtype=BF16, device="cuda")
    tl.tiled_linear_grouped_forward(R, K, n, E, 0, x.data_ptr(), K, R, None, w.data_ptr(), n, K * n, off.data_ptr(), y[:, 8:].data_ptr(), n + 16, None, 0, err, s)
    tl.tiled_linear_grouped_dw(R, K, n, E, 0, x.data_ptr(), K, R, None, dy.data_ptr(), n, off.data_ptr(), dw.data_ptr(), n + 8, (K + 1) * (n + 8), None, 0, err, s)
    check("y", y[:, 8:8 + n], *grouped(x, w, off))
    check("dw", dw[:, :K, :n], *grouped_backward(x, dy, w, off)[1])
    assert (y[:, :8] == 7).all() and (y[:, 8 + n:] == 7).all() and (dw[:, K:] == 7).all() and (dw[:, :, n:] == 7).all()


def test_indices_and_offsets_outside(tl):
    """Rows outside x count as zeros, places past R are left out, offsets that fall hold no rows."""
    K, n, R = 128, 384, 300
    x, w, dy = normal(1, 50, K), normal(2, 3, K, n), normal(3, R, n)
    rows = indices(4, R, 50)
    rows[::7] = 50 + torch.arange(len(rows[::7]), device="cuda").int()
    rows[3::50] = -1
    rows[4::90] = 2 ** 31 - 1
    off = torch.tensor([0, 100, 120, 5000], dtype=torch.int32, device="cuda")
    padded = torch.cat([x, torch.zeros(1, K, dtype=BF16, device="cuda")])
    inside = torch.where((rows >= 0) & (rows < 50), rows, 50)
    clipped = torch.tensor([0, 100, 120, R], dtype=torch.int32, device="cuda")
    check("y", tl.grouped_linear(x, w, off, rows), *grouped(padded, w, clipped, inside))
    for name, a, ref in zip(("dx", "dw"), tl.grouped_linear_backward(x, dy, w, off, rows), grouped_backward(padded, dy, w, clipped, inside)):
        check(name, a, *ref)
    for odd in ([5, 300, 10, 200], [-7, 50, 50, 300], [2 ** 31 - 1, 0, -2 ** 31, 7]):
        tl.grouped_linear(x, w, torch.tensor(odd, dtype=torch.int32, device="cuda"), rows)
        tl.grouped_linear_backward(x, dy, w, torch.tensor(odd, dtype=torch.int32, device="cuda"), rows)
    torch.cuda.synchronize()


@pytest.mark.parametrize("most", [40, 3])
def test_as_many_groups_as_there_may_be(tl, most):
    g = torch.Generator().manual_seed(most)
    both(tl, torch.randint(0, most, (1024,), generator=g).tolist(), 72, 136, BF16, True)


def test_many_rows_and_none_in_a_group(tl):
    """Offsets that hold nothing, where the sizes alone ask for the kernels of many rows."""
    x, w, dy = normal(1, 300, 64), normal(2, 2, 64, 264), normal(3, 300, 264)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    y = torch.full((300, 264), 7.0, dtype=BF16, device="cuda")
    s, err = torch.cuda.current_stream().cuda_stream, tl.tiled_linear_operator_error_word()
    tl.tiled_linear_grouped_forward(300, 64, 264, 2, 0, x.data_ptr(), 64, 300, None, w.data_ptr(), 264, 64 * 264, off.data_ptr(), y.data_ptr(), 264, None, 0, err, s)
    assert (y == 7).all()
    assert not tl.grouped_linear_backward(x, dy, w, off)[1].any()
    tl.check_operators()


def test_no_rows(tl):
    x, w, off = normal(1, 0, 64), normal(2, 3, 64, 200), torch.zeros(4, dtype=torch.int32, device="cuda")
    assert tl.grouped_linear(x, w, off).shape == (0, 200)
    dx, dw = tl.grouped_linear_backward(x, normal(1, 0, 200), w, off)
    assert dx.shape == (0, 64) and (dw == 0).all()
    x = normal(1, 10, 64)  # rows, all of no group
    dx, dw = tl.grouped_linear_backward(x, normal(1, 10, 200), w, off)
    assert (dw == 0).all()


def test_offsets_past_32_bits(tl):
    """Elements of weights and rows more than 2^31 away from the first."""
    K, n, E = 8192, 4096, 66
    w = torch.zeros(E, K, n, dtype=BF16, device="cuda")
    w[-1] = normal(1, K, n)
    counts = [0] * (E - 1) + [5]
    off, x = offsets_of(counts), normal(2, 5, K)
    check("y", tl.grouped_linear(x, w, off), *grouped(x, w[-1:], off[-2:] * 1))
    dy = normal(3, 5, n)
    dx, dw = tl.grouped_linear_backward(x, dy, w, off)
    (rx, rw) = grouped_backward(x, dy, w[-1:], off[-2:] * 1)
    check("dx", dx, *rx)
    check("dw", dw[-1:], *rw)
    assert not dw[:-1].any()
    del w, dw
    T = 2 ** 31 // 1024 + 500
    big = torch.zeros(T, 1024, dtype=BF16, device="cuda")
    rows = torch.tensor([T - 1, T - 400, 3], dtype=torch.int32, device="cuda").repeat(100)
    big[T - 1], big[T - 400] = normal(4, 1024), normal(5, 1024)
    w, off = normal(6, 2, 1024, 264), offsets_of([150, 150])
    small, at = big[[T - 1, T - 400, 3]], torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda").repeat(100)
    check("y", tl.grouped_linear(big, w, off, rows), *grouped(small, w, off, at))
    check("dw", tl.grouped_linear_backward(big, normal(7, 300, 264), w, off, rows)[1], *grouped_backward(small, normal(7, 300, 264), w, off, at)[1])


@pytest.mark.parametrize("counts,K,n", [([5, 0, 9], 2048, 512), ([300, 0, 190], 320, 520)])
def test_gradients_by_differences(tl, counts, K, n):
    """The product's change along a direction, in 64 bits, against what dx and dw say of it: it is bilinear, so the
    central difference with a step of one is exact."""
    off, R = offsets_of(counts), sum(counts)
    x, w, g = normal(1, R, K), normal(2, 3, K, n), normal(3, R, n)
    vx, vw = normal(4, R, K).double(), normal(5, 3, K, n).double()
    (dx, dw), ((rx, bx), (rw, bw)) = tl.grouped_linear_backward(x, g, w, off), grouped_backward(x, g, w, off)

    def total(e):
        y = 0.0
        for i, a in enumerate(counts):
            s = slice(off[i].item(), off[i].item() + a)
            y = y + (((x[s].double() + e * vx[s]) @ (w[i].double() + e * vw[i])) * g[s].double()).sum()
        return y

    slope = (total(1.0) - total(-1.0)) / 2
    assert abs((dx.double() * vx).sum() + (dw.double() * vw).sum() - slope) <= (bx * vx.abs()).sum() + (bw * vw.abs()).sum()


@pytest.mark.parametrize("T,E,k,K,n", [(6, 8, 2, 1024, 512), (300, 8, 2, 256, 640)])
def test_same_bits_again_and_together(tl, T, E, k, K, n):
    """Calls on two streams at once, and a captured one replayed with other inputs: the bits of calls alone."""
    logits = [normal(s, T, E) for s in range(3)]
    x, dy = [normal(s + 3, T, K) for s in range(3)], [normal(s + 6, T * k, n) for s in range(3)]
    w = normal(9, E, K, n)

    def call(l, a, d):
        weights, _, slots, rows, off = tl.route(l, k)
        y = tl.grouped_linear(a, w, off, rows)
        dx, dw = tl.grouped_linear_backward(a, d, w, off, rows)
        return y, dw, tl.combine(y, slots, weights), tl.combine(dx, slots)

    want = [call(*a) for a in zip(logits, x, dy)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(20):
        with torch.cuda.stream(streams[i % 2]):
            got.append(call(logits[i % 3], x[i % 3], dy[i % 3]))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[i % 3])), i
    held = [t.clone() for t in (logits[0], x[0], dy[0])]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(*held)
    for i in (0, 1, 2):
        for t, s in zip(held, (logits[i], x[i], dy[i])):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i])), i
