"""The operators around the product in company: calls in flight together, on several streams, in graphs, and after one
another without a pause."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tl():
    import __graft_entry__ as g
    g.build()
    from offload_streamed_gb300 import tiled_linear
    yield tiled_linear
    tiled_linear.check_operators()


def normal(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("batch,rows,cols", [(1, 64, 512), (1, 256, 1024), (4, 200, 520), (2, 256, 2048)])
def test_small_updates_in_a_row(tl, batch, rows, cols):
    """Chains of launches whose clusters share reductions, on two streams at once, each launch beginning while the one
    before it ends: every call gives the bits of a call alone."""
    g = [normal(s, batch, rows, cols) for s in range(3)]
    want = [tl.orthogonalize(m) for m in g]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(30):
        with torch.cuda.stream(streams[i % 2]):
            got.append(tl.orthogonalize(g[i % 3]))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % 3]), i


@pytest.mark.parametrize("T,K,n", [(1, 1024, 4096), (5, 8192, 1000), (64, 4096, 520), (128, 2048, 392)])
def test_few_tokens_in_a_row(tl, T, K, n):
    """The few-token product, whose clusters share a reduction, on two streams at once: every call gives the bits of a
    call alone, and so does the gradient by the tokens."""
    x, dy = [normal(s, T, K) for s in range(3)], [normal(s + 9, T, n) for s in range(3)]
    w = [tl.fp8_quantize(normal(s + 3, K, n), "tile") for s in range(3)]
    want = [(tl.fp8_linear(a, *b), tl.fp8_matmul_dx(tl.fp8_quantize(d, "row"), b)) for a, b, d in zip(x, w, dy)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(60):
        with torch.cuda.stream(streams[i % 2]):
            got.append((tl.fp8_linear(x[i % 3], *w[i % 3]), tl.fp8_matmul_dx(tl.fp8_quantize(dy[i % 3], "row"), w[i % 3])))
    torch.cuda.synchronize()
    for i, (y, dx) in enumerate(got):
        assert torch.equal(y, want[i % 3][0]) and torch.equal(dx, want[i % 3][1]), i
