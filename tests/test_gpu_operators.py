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
