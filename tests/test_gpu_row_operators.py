"""The operators whose weight depends on the row in company: a layer of them as it is trained and served, a process's first
call captured in a graph, calls with the error word set, two threads."""
import os
import subprocess
import sys
import threading

import pytest
import torch

from rows_reference import STEP, half
from test_gpu_operators import FIRST_CALL

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


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


class Layer:
    """x -> y0 = x . W (streamed from host memory) -> y1 = y0 + the request's adapter -> the two best of E experts' answers
    to y1, weighted and summed; forward and backward by the package."""

    def __init__(self, tl, K=512, n=512, m=384, E=6, k=2, r=16, R=3, seed=1):
        self.tl, self.k, self.E = tl, k, E
        self.w, self.dw = tl.PinnedBuffer(K * n), tl.PinnedBuffer(K * n)
        self.w.tensor.copy_((normal(seed, 2, K, n // 2) / K ** 0.5).cpu().reshape(-1))
        self.op = tl.TiledLinear(K, n, 2, 1, self.w, self.dw)
        self.a, self.b = normal(seed + 1, R, K, r) / K ** 0.5, normal(seed + 2, R, r, n) / r ** 0.5
        self.scale = torch.tensor([0.5, 1.0, 2.0], device="cuda")
        self.router, self.experts = normal(seed + 3, n, E) / n ** 0.5, normal(seed + 4, E, n, m) / n ** 0.5

    def forward(self, x, ids):
        tl, c = self.tl, {"x": x, "ids": ids}
        base = self.op.forward(x)
        c["y1"], c["h"] = tl.adapter_linear(x, self.a, self.b, ids, base=base, scale=self.scale)
        c["logits"] = c["y1"] @ self.router
        c["weights"], c["chosen"], c["slots"], c["rows"], c["offsets"] = tl.route(c["logits"], self.k)
        c["u"] = tl.grouped_linear(c["y1"], self.experts, c["offsets"], c["rows"])
        return tl.combine(c["u"], c["slots"], c["weights"]), c

    def backward(self, dout, c):
        tl = self.tl
        du, dweights = tl.combine_backward(dout, c["slots"], c["u"], c["weights"])
        dsorted, dexperts = tl.grouped_linear_backward(c["y1"], du, self.experts, c["offsets"], c["rows"])
        dlogits = tl.route_backward(dweights, c["logits"], c["chosen"])
        dy1 = (tl.combine(dsorted, c["slots"]).float() + dlogits.float() @ self.router.float().T).to(BF16)
        dbase = self.op.backward(c["x"], dy1)  # fp32; dW in host memory
        dx, da, db = tl.adapter_linear_backward(c["x"], c["h"], dy1, self.a, self.b, c["ids"], base=dbase, scale=self.scale)
        return dx, da, db, dexperts

    def exact(self, x, ids, chosen, dout):
        """The same in 64 bits by automatic differentiation, with the package's choice of experts."""
        K, n = self.op.K, self.op.M
        leaf = lambda t: t.double().detach().requires_grad_(True)  # noqa: E731
        x, a, b, ex = leaf(x), leaf(self.a), leaf(self.b), leaf(self.experts)
        W = self.w.tensor.cuda().reshape(2, K, n // 2).permute(1, 0, 2).reshape(K, n).double()
        y1 = x @ W
        for i in range(a.shape[0]):
            own = (ids == i).double()[:, None]
            y1 = y1 + own * float(self.scale[i]) * ((x @ a[i]) @ b[i])
        weights = torch.softmax((y1 @ self.router.double()).gather(1, chosen.long()), 1)
        out = 0.0
        for j in range(self.k):
            for e in range(self.E):
                out = out + (chosen[:, j] == e).double()[:, None] * weights[:, j, None] * (y1 @ ex[e])
        (out * dout.double()).sum().backward()
        return out.detach(), x.grad, a.grad, b.grad, ex.grad

    def close(self):
        self.op.close()
        self.w.close()
        self.dw.close()


@pytest.mark.parametrize("T", [5, 700])
def test_a_layer_trained_and_served(tl, T):
    """Every intermediate tensor is rounded to bf16 (half a step: 2^-8, 2^-8 / sqrt(3) of it in the mean); a result has at
    most eight of those in its path (x . W, the adapter, logits, answers, the sum, and their gradients), which add up as
    sqrt(8) of one where they are independent and as eight where they are not: 8 * 2^-8 / sqrt(3) of its norm."""
    layer = Layer(tl)
    x, dout = normal(11, T, 512), normal(12, T, 384)
    ids = torch.randint(-1, 3, (T,), generator=torch.Generator().manual_seed(4), dtype=torch.int32).cuda()
    out, c = layer.forward(x, ids)
    got = layer.backward(dout, c)
    torch.cuda.synchronize()
    tl.check_operators()
    ref = layer.exact(x, ids, c["chosen"], dout)
    for name, g, e in zip(("out", "dx", "da", "db", "dexperts"), (out, *got), ref):
        err = ((g.double() - e).norm() / e.norm()).item()
        assert err <= 8 * half(BF16) / 3 ** 0.5, f"{name}: {err:.3g}"
    # served a token at a time: the same answers where the same experts are chosen
    for t in range(min(T, 4)):
        one, c1 = layer.forward(x[t:t + 1].contiguous(), ids[t:t + 1].contiguous())
        if torch.equal(c1["chosen"][0], c["chosen"][t]):
            err = ((one.double() - ref[0][t:t + 1]).norm() / ref[0][t].norm()).item()
            assert err <= 8 * half(BF16) / 3 ** 0.5, err
    layer.close()


CALLS = {
    "route": "lambda x: tl.route(x, 3)",
    "group_rows": "lambda x: tl.group_rows((x[:, :2] * 3).int(), 4)",
    "combine": "lambda x: (tl.combine(x, torch.arange(40, dtype=torch.int32, device='cuda').reshape(20, 2)),)",
    "grouped": "lambda x: (tl.grouped_linear(x, wide, off),)",
    "grouped_backward": "lambda x: tl.grouped_linear_backward(x, x[:, :512], wide, off, torch.arange(40, dtype=torch.int32, device='cuda'))",
    "adapter": "lambda x: tl.adapter_linear(x, wide[:, :, :16], wide[:, :16], torch.arange(40, dtype=torch.int32, device='cuda') % 3)",
    "adapter_backward": "lambda x: tl.adapter_linear_backward(x, x[:, :16], x[:, :512], wide[:, :, :16], wide[:, :16], "
                        "torch.arange(40, dtype=torch.int32, device='cuda') % 3)",
}


@pytest.mark.parametrize("call", CALLS)
def test_first_call_in_a_graph(tl, call):
    """A process's first call of an operator may be captured, and replays with other inputs."""
    src = FIRST_CALL.format(root=os.path.dirname(os.path.dirname(os.path.abspath(__file__))), call=CALLS[call])
    src = src.replace("call = lambda", "wide = normal(4, 2, 1024, 512)\noff = torch.tensor([0, 30, 40], dtype=torch.int32, device='cuda')\ncall = lambda", 1)
    if call == "group_rows":  # (its first result may be the same for both inputs)
        src = src.replace("and not torch.equal(got[0], first[0])", "")
    r = subprocess.run([sys.executable, "-c", src], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def calls_of(tl):
    T, K, n, E = 300, 256, 320, 5
    x, dy, w = normal(1, T, K), normal(2, 2 * T, n), normal(3, E, K, n)
    a, b, ids = normal(4, 3, K, 16), normal(5, 3, 16, n), (torch.arange(T, device="cuda") % 4).int()
    weights, chosen, slots, rows, off = tl.route(normal(6, T, E), 2)

    def run():
        y = tl.grouped_linear(x, w, off, rows)
        few = tl.grouped_linear(x[:8], w, (off // 100).int())
        z, h = tl.adapter_linear(x, a, b, ids)
        return (y, few[:off[-1].item() // 100], z, h, tl.combine(y, slots, weights), *tl.grouped_linear_backward(x, dy, w, off, rows),
                *tl.adapter_linear_backward(x, h, dy[:T], a, b, ids), *tl.adapter_linear(x[:7], a, b, ids[:7]))
    return run


def test_a_word_that_is_set_already(tl):
    """What an earlier call has left in the error word ends no later call's waits; check_operators reports and clears it."""
    run = calls_of(tl)
    want = run()
    tl.check_operators()
    tl._err_words[torch.cuda.current_device()][0][0] = 1 << 20
    got = run()
    with pytest.raises(tl.TiledLinearError) as e:
        tl.check_operators()
    assert e.value.status == tl.TL_ERR_TIMEOUT and hex(1 << 20) in str(e.value)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_two_threads(tl):
    run = calls_of(tl)
    want = run()
    torch.cuda.synchronize()
    bad, device = [], torch.cuda.current_device()

    def loop():
        torch.cuda.set_device(device)
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(15):
                got = run()
                s.synchronize()
                bad.extend(i for i, (p, q) in enumerate(zip(got, want)) if not torch.equal(p, q))

    threads = [threading.Thread(target=loop) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
        assert not t.is_alive()
    assert not bad, bad


def test_graphs_that_replay_at_once(tl):
    """Two captured calls replayed on two streams at the same time: each has its own workspace."""
    xs = [normal(s, 600, 256) for s in (1, 2)]
    a, b, ids = normal(4, 3, 256, 32), normal(5, 3, 32, 320), (torch.arange(600, device="cuda") // 7 % 4 - 1).int()
    w, logits = normal(6, 5, 256, 320), [normal(s, 600, 5) for s in (7, 8)]

    def call(x, l):
        weights, _, slots, rows, off = tl.route(l, 2)
        y = tl.grouped_linear(x, w, off, rows)
        return tl.combine(y, slots, weights), *tl.adapter_linear(x, a, b, ids)

    want = [call(x, l) for x, l in zip(xs, logits)]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for x, l in zip(xs, logits):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(x, l))
        graphs.append(g)
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, v in zip(outs, want):
        assert all(torch.equal(p, q) for p, q in zip(o, v))


def test_other_devices_and_shapes_are_refused(tl):
    x, w, off = normal(1, 10, 64), normal(2, 2, 64, 32), torch.tensor([0, 4, 10], dtype=torch.int32, device="cuda")
    ids = torch.zeros(10, dtype=torch.int32, device="cuda")
    a, b = normal(3, 2, 64, 8), normal(4, 2, 8, 32)
    bad = [lambda: tl.grouped_linear(x, w.half(), off), lambda: tl.grouped_linear(x, w, off.cpu()), lambda: tl.grouped_linear(x, w, off[:2]),
           lambda: tl.grouped_linear(x, w, off.long()), lambda: tl.grouped_linear(x[:, :32], w, off), lambda: tl.grouped_linear(x, w, off, ids[None]),
           lambda: tl.grouped_linear(x, w.transpose(1, 2), off), lambda: tl.grouped_linear(x, w[:1].expand(2, 64, 32), off),
           lambda: tl.grouped_linear_backward(x, x, w, off), lambda: tl.adapter_linear(x, a, b, ids[:5]), lambda: tl.adapter_linear(x, b, a, ids),
           lambda: tl.adapter_linear(x, a, b, ids, base=x), lambda: tl.adapter_linear(x, a, b, ids, scale=torch.ones(3, device="cuda")),
           lambda: tl.adapter_linear(x, a, b, ids, base=normal(5, 10, 32, dtype=torch.float16)), lambda: tl.adapter_linear_backward(x, x, x, a, b, ids),
           lambda: tl.route(x, 0), lambda: tl.route(x, 65), lambda: tl.route(x, 33), lambda: tl.group_rows(ids, 4), lambda: tl.group_rows(ids[:, None], 0),
           lambda: tl.group_rows(ids[:, None], 1025), lambda: tl.combine(x, ids), lambda: tl.combine(x, ids[:, None], x),
           lambda: tl.combine_backward(x, ids[:5, None]), lambda: tl.route_backward(x, x, ids[:, None])]
    for i, f in enumerate(bad):
        with pytest.raises(tl.TiledLinearError) as e:
            f()
        assert e.value.status in (tl.TL_ERR_INVALID, tl.TL_ERR_WORKSPACE), (i, e.value)
    assert STEP == 2.0 ** -23
