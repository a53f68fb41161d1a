"""The operators around the product in company: calls in flight together, on several streams, in graphs, and after one
another without a pause."""
import os
import subprocess
import sys
import threading

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


def test_a_word_that_is_set_already(tl):
    """The error word is shared by all calls: what an earlier one has left in it ends no later call's waits, however
    long (one output tile here sums over 8 million tokens), and check_operators reports and clears it."""
    T, K, n = 65535 * 128, 16, 16
    x, dy = (normal(s, T, 16) for s in (1, 2))
    xc, dyc = tl.fp8_quantize(x, "col"), tl.fp8_quantize(dy, "col")
    row = tl.fp8_quantize(dy[:64, :16].contiguous(), "row")
    w = tl.fp8_quantize(normal(3, K, n), "tile")
    g = normal(4, 2, 256, 1024)
    calls = [lambda: tl.fp8_matmul_dw(xc, dyc), lambda: tl.fp8_matmul_dx(row, w), lambda: tl.orthogonalize(g),
             lambda: tl.layer_norm(x)[0]]
    want = [c() for c in calls]
    tl.check_operators()
    word = tl._err_words[x.device.index][0]
    word[0] = 1 << 20
    out = torch.full((1 << 20,), float("nan"), device="cuda")  # what a freed result may hold
    del out
    got = [c() for c in calls]
    with pytest.raises(tl.TiledLinearError) as e:
        tl.check_operators()
    assert e.value.status == tl.TL_ERR_TIMEOUT and hex(1 << 20) in str(e.value)
    tl.check_operators()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(c(), b) for c, b in zip(calls, want))


FIRST_CALL = """
import sys, torch
sys.path.insert(0, {root!r})
from offload_streamed_gb300 import tiled_linear as tl
normal = lambda s, *shape: torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(s), device="cuda").bfloat16()
x, other = normal(1, 40, 1024), normal(2, 40, 1024)
wq = normal(3, 1024, 512).to(torch.float8_e4m3fn)
ws = torch.full((8, 4), 127, dtype=torch.uint8, device="cuda")
mean, rstd = torch.zeros(40, device="cuda"), torch.ones(40, device="cuda")
call = {call}
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = call(x)
g.replay()
first = [t.clone() for t in got]
want = call(x)
assert all(torch.equal(a, b) for a, b in zip(first, want))
x.copy_(other)
g.replay()
want = call(other)
assert all(torch.equal(a, b) for a, b in zip(got, want)) and not torch.equal(got[0], first[0])
tl.check_operators()
print("captured")
"""


@pytest.mark.parametrize("call", ["lambda x: tl.layer_norm(x)", "lambda x: tl.layer_norm_backward(x, x, mean, rstd)",
                                  "lambda x: (tl.fp8_linear(x, wq, ws),)", "lambda x: tl.fp8_linear_backward(x, x[:, :512], wq, ws)",
                                  "lambda x: tl.fp8_quantize(x, 'row')", "lambda x: (tl.orthogonalize(x),)"])
def test_first_call_in_a_graph(tl, call):
    """A process's first call of an operator may be captured, and replays with other inputs."""
    src = FIRST_CALL.format(root=os.path.dirname(os.path.dirname(os.path.abspath(__file__))), call=call)
    r = subprocess.run([sys.executable, "-c", src], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_two_threads(tl):
    """Calls from two threads, each on a stream of its own, at the same time: the bits of calls alone."""
    x, dy, w = normal(1, 70, 1024), normal(2, 70, 512), normal(3, 1024, 512)
    stack = normal(4, 3, 120, 260)

    def calls():
        y, mean, rstd = tl.layer_norm(x)
        wq, ws = tl.fp8_quantize(w, "tile")
        return (y, *tl.layer_norm_backward(x, x, mean, rstd), tl.fp8_linear(y, wq, ws), *tl.fp8_linear_backward(y, dy, wq, ws),
                tl.orthogonalize(stack))

    want = calls()
    torch.cuda.synchronize()
    bad, device = [], torch.cuda.current_device()

    def run():
        torch.cuda.set_device(device)
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                got = calls()
                s.synchronize()
                bad.extend(i for i, (a, b) in enumerate(zip(got, want)) if not torch.equal(a, b))

    threads = [threading.Thread(target=run) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
        assert not t.is_alive()
    assert not bad, bad
