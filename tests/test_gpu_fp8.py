"""The 8-bit forms and products (through the package's functions, so through the
C ABI) against their definition.

The forms are exact: values and scale bytes have to be equal to those that a
plain implementation in 64 bits gives.  The products are compared with the
64-bit product of the values that the forms stand for, within gpu_check's
bound: products of two 4-bit significands are exact in fp32, so only the fp32
sum (gamma_K of the sum of magnitudes, with its slack for a tensor core that
truncates) and the rounding to bf16 are in it."""
import numpy as np
import pytest
import torch

from gpu_check import check

pytestmark = pytest.mark.gpu

FORMATS = {"e4m3": (3, -6, 448.0), "e5m2": (2, -14, 57344.0)}  # significand bits after the first, least exponent, top
BLOCKS = {"row": (1, 128), "col": (128, 1), "tile": (128, 128)}


@pytest.fixture(scope="module")
def tl():
    import __graft_entry__ as g
    g.build()
    from offload_streamed_gb300 import tiled_linear
    yield tiled_linear
    tiled_linear.check_operators()


def reference(x: np.ndarray, form: str, fmt: str):
    """(values that the form stands for, scale bytes) of x, in 64 bits."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    br, bc = BLOCKS[form]
    bits, least, top = FORMATS[fmt]
    out, scale = np.zeros_like(x), np.zeros((-(-rows // br), -(-cols // bc)), np.uint8)
    for i in range(scale.shape[0]):
        for j in range(scale.shape[1]):
            at = (slice(i * br, (i + 1) * br), slice(j * bc, (j + 1) * bc))
            blk = x[at]
            if not np.isfinite(blk).all():
                scale[i, j], out[at] = 255, np.nan
                continue
            amax = np.abs(blk).max()
            e = 0
            if amax > 0:
                e = -127
                while amax > top * 2.0 ** e:
                    e += 1
            scale[i, j] = e + 127
            v = blk / 2.0 ** e
            ex = np.maximum(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -300))), least)
            step = 2.0 ** (ex - bits)
            out[at] = np.rint(v / step) * step * 2.0 ** e
    return out, scale


def plain_scales(scale, rows, cols, form):
    """The bytes as [rows, cols / 128], [rows / 128, cols] or [rows / 128, cols / 128]; those past
    the last block of a word have to be 127."""
    s = scale.cpu().numpy()
    if form == "tile":
        return s
    s = s.transpose(1, 0, 2).reshape(s.shape[1], -1)  # [vector, block]
    have = -(-(cols if form == "row" else rows) // 128)
    assert (s[:, have:] == 127).all()
    return s[:, :have] if form == "row" else s[:, :have].T


def packed(s, form):
    """The inverse, as a device tensor."""
    v = s.numpy() if form == "row" else s.numpy().T
    v = np.pad(v, ((0, 0), (0, -v.shape[1] % 4)), constant_values=127)
    return torch.from_numpy(np.ascontiguousarray(v.reshape(v.shape[0], -1, 4).transpose(1, 0, 2))).cuda()


def values(q, scale, form):
    br, bc = BLOCKS[form]
    rows, cols = q.shape
    e = plain_scales(scale, rows, cols, form).astype(np.int64)
    s = np.where(e == 255, np.nan, 2.0 ** (e - 127.0))
    s = np.repeat(np.repeat(s, br, 0)[:rows], bc, 1)[:, :cols]
    return q.cpu().float().numpy().astype(np.float64) * s


def make(rows, cols, seed, dtype=torch.bfloat16, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(spread * torch.randn(rows, 1, generator=g))
    return (x * torch.exp(0.5 * torch.randn(1, cols, generator=g))).to(dtype)


@pytest.mark.parametrize("fmt", list(FORMATS))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 4096), (3, 127), (128, 128), (130, 264), (257, 1000), (300, 72)])
def test_forms_are_exact(tl, rows, cols, dtype, fmt):
    x = make(rows, cols, rows + cols, dtype)
    x[0, : cols // 2] = 0
    got = tl.fp8_quantize(x.cuda(), "tile", "row", "col", format=fmt)
    for (q, s), form in zip(got, ("tile", "row", "col")):
        ref, sref = reference(x.double().numpy(), form, fmt)
        assert np.array_equal(plain_scales(s, rows, cols, form), sref), form
        assert np.array_equal(values(q, s, form), ref, equal_nan=True), form
        one, sone = tl.fp8_quantize(x.cuda(), form, format=fmt)  # a form alone is the same
        assert torch.equal(sone, s) and torch.equal(one.view(torch.uint8), q.view(torch.uint8))


def test_forms_at_the_edges(tl):
    """Ties, the largest values, subnormal blocks, zeros, NaN and infinities."""
    x = torch.zeros(9, 256)
    x[0, 0], x[0, 1:17] = 448.0, torch.arange(16) + 0.5            # ties between whole steps
    x[1, 0], x[1, 1] = 448.0001, 1.0                                # just over the top: the next scale
    x[2, :128] = 2.0 ** -130                                        # subnormal in fp32
    x[3, 0], x[3, 1] = 3.0e38, -1.0e30
    x[4, 5] = float("nan")
    x[5, 130] = float("inf")
    x[6, :] = -0.0
    x[7, 0], x[7, 1] = 1.0, 2.0 ** -12                              # under the format's least step
    x[8, 0], x[8, 1:9] = 256.0, torch.tensor([17.0, 19.0, 21.0, 23.0, 25.0, 27.0, 29.0, 31.0])
    for form in ("row", "col"):
        y = x if form == "row" else x.T.contiguous()
        q, s = tl.fp8_quantize(y.cuda(), form)
        ref, sref = reference(y.numpy(), form, "e4m3")
        assert np.array_equal(plain_scales(s, *y.shape, form), sref)
        assert np.array_equal(values(q, s, form), ref, equal_nan=True)


@pytest.mark.parametrize("ld,off", [(264, 8), (261, 0), (261, 3)])
def test_forms_of_strided_rows(tl, ld, off):
    x = make(70, 200, 4)
    buf = torch.full((70, ld), float("nan"), dtype=torch.bfloat16, device="cuda")
    xd = torch.as_strided(buf, (70, 200), (ld, 1), off)
    xd.copy_(x)
    q, s = tl.fp8_quantize(xd, "row")
    ref, sref = reference(x.double().numpy(), "row", "e4m3")
    assert np.array_equal(plain_scales(s, 70, 200, "row"), sref) and np.array_equal(values(q, s, "row"), ref)


def compare(name, got, a, b, K):
    """got against a [M, K] . b [K, N] in 64 bits (on the GPU: the sizes are not small)."""
    a, b = torch.from_numpy(a).cuda(), torch.from_numpy(b).cuda()
    check(name, got.float().cpu().numpy(), (a @ b).cpu().numpy(), (a.abs() @ b.abs()).cpu().numpy(), K, bf16_out=True)


# from one token to several tiles in each direction; ragged in each; reductions of one block to many,
# not whole chunks of four blocks; enough tiles that a CTA pair has several
SHAPES = [(1, 128, 128), (1, 1, 1), (2, 64, 40), (16, 1024, 512), (17, 130, 260), (33, 640, 72), (64, 2048, 1000),
          (65, 513, 300), (100, 384, 1032), (128, 4096, 256), (129, 1000, 520), (256, 256, 256), (300, 1160, 776),
          (517, 1032, 264), (1024, 896, 5128), (2500, 512, 4100)]


@pytest.mark.parametrize("T,K,n", SHAPES)
def test_linear_and_its_gradients(tl, T, K, n):
    x, w, dy = make(T, K, 1, spread=1.0), make(K, n, 2, spread=0.2), make(T, n, 3, spread=2.0)
    xd, wd, dyd = x.cuda(), w.cuda(), dy.cuda()
    wq, ws = tl.fp8_quantize(wd, "tile")
    wv = values(wq, ws, "tile")
    y = tl.fp8_linear(xd, wq, ws)
    xr = reference(x.double().numpy(), "row", "e4m3")[0] if T * K < 300000 else values(*tl.fp8_quantize(xd, "row"), "row")
    compare("y", y, xr, wv, K)
    dx, dw = tl.fp8_linear_backward(xd, dyd, wq, ws)
    compare("dx", dx, values(*tl.fp8_quantize(dyd, "row"), "row"), np.ascontiguousarray(wv.T), n)
    compare("dw", dw, np.ascontiguousarray(values(*tl.fp8_quantize(xd, "col"), "col").T),
            values(*tl.fp8_quantize(dyd, "col"), "col"), T)


@pytest.mark.parametrize("T", [8, 200])
@pytest.mark.parametrize("fx,fw", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
def test_formats_mix(tl, T, fx, fw):
    x, w, dy = make(T, 700, 1, spread=1.0), make(700, 300, 2, spread=0.2), make(T, 300, 3)
    a, b = tl.fp8_quantize(x.cuda(), "row", format=fx), tl.fp8_quantize(w.cuda(), "tile", format=fw)
    compare("y", tl.fp8_matmul(a, b), values(*a, "row"), values(*b, "tile"), 700)
    g = tl.fp8_quantize(dy.cuda(), "row", format=fx)
    compare("dx", tl.fp8_matmul_dx(g, b), values(*g, "row"), np.ascontiguousarray(values(*b, "tile").T), 300)
    xc, gc = tl.fp8_quantize(x.cuda(), "col", format=fw), tl.fp8_quantize(dy.cuda(), "col", format=fx)
    compare("dw", tl.fp8_matmul_dw(xc, gc), np.ascontiguousarray(values(*xc, "col").T), values(*gc, "col"), T)


@pytest.mark.parametrize("T", [4, 300])
def test_every_scale_is_applied(tl, T):
    """Ones in every block and a power of two of its own for each: sums are exact
    (products of 32 ones lie between 2^-7 and 2^11, their sums under 2^16: 23 bits),
    so a scale that is off by one row, column or block shows."""
    K, n = 1280, 640
    g = torch.Generator().manual_seed(9)
    xs = torch.randint(120, 132, (T, K // 128), generator=g, dtype=torch.uint8)
    ws = torch.randint(122, 130, (K // 128, n // 128), generator=g, dtype=torch.uint8)
    one = lambda r, c: torch.ones(r, c).to(torch.float8_e4m3fn).cuda()  # noqa: E731
    y = tl.fp8_matmul((one(T, K), packed(xs, "row")), (one(K, n), ws.cuda()))
    ref = (2.0 ** (xs.double() - 127)) @ (2.0 ** (ws.double() - 127)) * 128
    assert torch.equal(y.cpu(), ref.repeat_interleave(128, 1).bfloat16())
    gs = torch.randint(120, 132, (T, n // 128), generator=g, dtype=torch.uint8)
    dx = tl.fp8_matmul_dx((one(T, n), packed(gs, "row")), (one(K, n), ws.cuda()))
    ref = (2.0 ** (gs.double() - 127)) @ (2.0 ** (ws.double().T - 127)) * 128
    assert torch.equal(dx.cpu(), ref.repeat_interleave(128, 1).bfloat16())
    tb = -(-T // 128)
    xc = torch.randint(120, 132, (tb, K), generator=g, dtype=torch.uint8)
    gc = torch.randint(122, 130, (tb, n), generator=g, dtype=torch.uint8)
    dw = tl.fp8_matmul_dw((one(T, K), packed(xc, "col")), (one(T, n), packed(gc, "col")))
    count = torch.tensor([min(128, T - 128 * i) for i in range(tb)], dtype=torch.float64)
    ref = (2.0 ** (xc.double().T - 127) * count) @ (2.0 ** (gc.double() - 127))
    assert torch.equal(dw.cpu(), ref.bfloat16())


@pytest.mark.parametrize("T", [5, 260])
def test_nan_and_inf_stay_in_their_rows(tl, T):
    x, w = make(T, 600, 1, spread=1.0), make(600, 200, 2, spread=0.2)
    wq, ws = tl.fp8_quantize(w.cuda(), "tile")
    want = tl.fp8_linear(x.cuda(), wq, ws)
    x[1, 300], x[T - 1, 599] = float("nan"), float("inf")
    y = tl.fp8_linear(x.cuda(), wq, ws)
    bad = torch.zeros(T, dtype=torch.bool)
    bad[1] = bad[T - 1] = True
    assert torch.isnan(y[bad.cuda()]).all() and torch.equal(y[~bad.cuda()], want[~bad.cuda()])


@pytest.mark.parametrize("T,K,n", [(3, 256, 1024), (300, 512, 768)])
def test_gradients_against_differences(tl, T, K, n):
    """dx and dw are the derivatives of the layer without its rounding, so they are compared with
    differences of the unrounded layer (which is linear: the difference is exact) within the
    rounding of 8 bits, 2^-4 of each product at most."""
    x, w, dy = make(T, K, 1, spread=0.0), make(K, n, 2, spread=0.0), make(T, n, 3, spread=0.0)
    wq, ws = tl.fp8_quantize(w.cuda(), "tile")
    dx, dw = (t.double().cpu() for t in tl.fp8_linear_backward(x.cuda(), dy.cuda(), wq, ws))
    loss = lambda x, w: ((x @ w) * dy.double()).sum()  # noqa: E731
    x, w = x.double(), w.double()
    g = np.random.default_rng(1)
    for _ in range(10):
        t, k, j = int(g.integers(T)), int(g.integers(K)), int(g.integers(n))
        step = torch.zeros_like(x)
        step[t, k] = 1.0
        ref = (loss(x + step, w) - loss(x - step, w)).item() / 2
        # two rounded factors, each off by 2^-4 of itself or half a step of its block's least
        room = ((dy[t].double().abs() + 2.0 ** -9 * dy[t].abs().max()) * (w[k].abs() + 2.0 ** -9 * w.abs().max())).sum().item()
        assert abs(dx[t, k].item() - ref) <= 2.0 ** -3 * room + 1e-6
        step = torch.zeros_like(w)
        step[k, j] = 1.0
        ref = (loss(x, w + step) - loss(x, w - step)).item() / 2
        room = ((x[:, k].abs() + 2.0 ** -9 * x[:, k].abs().max()) * (dy[:, j].double().abs() + 2.0 ** -9 * dy[:, j].abs().max())).sum().item()
        assert abs(dw[k, j].item() - ref) <= 2.0 ** -3 * room + 1e-6


def test_no_tokens(tl):
    w = make(256, 128, 2)
    wq, ws = tl.fp8_quantize(w.cuda(), "tile")
    x, dy = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    assert tl.fp8_linear(x, wq, ws).shape == (0, 128)
    dx, dw = tl.fp8_linear_backward(x, dy, wq, ws)
    assert dx.shape == (0, 256) and dw.shape == (256, 128) and not dw.any()


@pytest.mark.parametrize("T", [2, 384])
def test_same_bits_and_another_stream(tl, T):
    x, w = make(T, 2000, 1, spread=1.0).cuda(), make(2000, 1000, 2, spread=0.2).cuda()
    wq, ws = tl.fp8_quantize(w, "tile")
    a = tl.fp8_linear(x, wq, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = tl.fp8_linear(x * 1, wq, ws)
    s.synchronize()
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("T", [3, 200])
def test_other_types_of_x_and_strides(tl, T, dtype):
    """The layer's one call gives what quantising and the products give, for every type and stride of x."""
    x, w, dy = make(T, 300, 1, dtype, spread=0.5), make(300, 200, 2, spread=0.2), make(T, 200, 3, dtype, spread=0.5)
    wq, ws = tl.fp8_quantize(w.cuda(), "tile")
    xd, dyd = torch.zeros(T, 333, dtype=dtype, device="cuda")[:, 5:305], torch.zeros(T, 211, dtype=dtype, device="cuda")[:, :200]
    xd.copy_(x)
    dyd.copy_(dy)
    assert torch.equal(tl.fp8_linear(xd, wq, ws), tl.fp8_matmul(tl.fp8_quantize(x.cuda(), "row"), (wq, ws)))
    dx, dw = tl.fp8_linear_backward(xd, dyd, wq, ws)
    row, col = tl.fp8_quantize(dy.cuda(), "row", "col")
    assert torch.equal(dx, tl.fp8_matmul_dx(row, (wq, ws)))
    assert torch.equal(dw, tl.fp8_matmul_dw(tl.fp8_quantize(x.cuda(), "col"), col))


def test_offsets_past_32_bits(tl):
    """More than 2^31 elements in x: the last rows' forms and products are theirs."""
    T, K, n = 34000, 65536, 128
    x = torch.empty(T, K, dtype=torch.bfloat16, device="cuda").normal_()
    wq, ws = tl.fp8_quantize(make(K, n, 2, spread=0.1).cuda(), "tile")
    y = tl.fp8_linear(x, wq, ws)
    few = tl.fp8_linear(x[-300:].clone(), wq, ws)
    assert torch.equal(y[-300:], few) or (y[-300:].float() - few.float()).norm() <= 2.0 ** -8 * few.float().norm()
    q, s = tl.fp8_quantize(x, "row")
    q1, s1 = tl.fp8_quantize(x[-2:].clone(), "row")
    assert torch.equal(q[-2:].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s[:, -2:], s1)


def test_refusals_of_the_functions(tl):
    """What does not fit is refused with a message before anything runs."""
    w = make(256, 128, 1).cuda()
    wq, ws = tl.fp8_quantize(w, "tile")
    x = make(4, 256, 2).cuda()
    for fn, words in ((lambda: tl.fp8_linear(x[:, :255], wq, ws), "fit"), (lambda: tl.fp8_linear(x, wq, ws[:, :0]), "scales"),
                      (lambda: tl.fp8_linear(x, wq.float(), ws), "float8"), (lambda: tl.fp8_linear(x.double(), wq, ws), "dtype"),
                      (lambda: tl.fp8_linear(x, wq[:, 1:], ws), "16-byte"), (lambda: tl.fp8_quantize(x, "rows"), "form"),
                      (lambda: tl.fp8_quantize(x), "form"), (lambda: tl.fp8_quantize(x, "row", format="e3m4"), "format"),
                      (lambda: tl.fp8_quantize(x.T, "row"), "contiguous"), (lambda: tl.fp8_linear(x.cpu(), wq, ws), "CUDA"),
                      (lambda: tl.fp8_matmul(tl.fp8_quantize(x, "col"), (wq, ws)), "scales"),
                      (lambda: tl.fp8_linear_backward(x, x, wq, ws), "fit")):
        with pytest.raises(tl.TiledLinearError) as e:
            fn()
        assert e.value.status == tl.TL_ERR_INVALID and words in str(e.value), e.value
