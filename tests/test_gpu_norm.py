"""Layer norm and its backward (through the package's functions, so through the
C ABI) against the formulas in 64 bits, and its gradients against differences.

Tolerances, u = 2^-24 (fp32) and v the rounding of the output's type
(2^-8 bf16, 2^-11 fp16, 2^-23 fp32, each one whole spacing):
 * a row's mean and variance come from sums of `cols` terms of fp32, joined
   pairwise: within 64 u of the terms' mean magnitude;
 * y and dx pass through about ten fp32 operations on values that are joined
   from such sums: within 64 u of the largest magnitude that goes into an
   element, plus v of the result;
 * a sum over `rows` terms: within (rows + 64) u of the sum of magnitudes
   (the sum is split over CTAs, so this is far from tight).
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
V = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -23}
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
# one column to the longest row of each kind: a warp's, a CTA's, a cluster's of
# each size, and the longest of all; vectors whole and ragged
SHAPES = [(1, 1), (3, 2), (1, 7), (5, 64), (37, 250), (64, 256), (33, 264), (9, 1000), (70, 1024), (6, 1025), (4, 1032),
          (300, 520), (13, 2048), (5, 5003), (40, 8192), (3, 8200), (2, 16384), (1, 25600), (3, 30001), (2, 65536),
          (2, 65544), (1, 131072), (1, 99999)]


@pytest.fixture(scope="module")
def tl():
    import __graft_entry__ as g
    g.build()
    from offload_streamed_gb300 import tiled_linear
    return tiled_linear


def make(rows, cols, dtype, seed, pdtype=None, mean=0.3, scale=1.7):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, cols, generator=g) * scale + mean).to(dtype)
    dy = torch.randn(rows, cols, generator=g).to(dtype)
    w = (1 + 0.2 * torch.randn(cols, generator=g)).to(pdtype or dtype)
    b = (0.3 * torch.randn(cols, generator=g)).to(pdtype or dtype)
    return x, dy, w, b


def forward64(x, w, b, eps):
    x = x.double()
    m = x.mean(1, keepdim=True)
    var = ((x - m) ** 2).mean(1, keepdim=True)
    r = 1 / torch.sqrt(var + eps)
    xh = (x - m) * r
    y = xh * (w.double() if w is not None else 1.0) + (b.double() if b is not None else 0.0)
    return y, m[:, 0], r[:, 0], xh


def backward64(dy, x, m, r, w):
    dy, x = dy.double(), x.double()
    m, r = m.double()[:, None], r.double()[:, None]
    xh = (x - m) * r
    g = dy * (w.double() if w is not None else 1.0)
    dx = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0), xh, g


def close(name, got, ref, bound):
    got = got.double().cpu()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert torch.isfinite(got).all(), name
    worst = ((got - ref).abs() / bound).max().item()
    assert worst <= 1.0, f"{name}: {worst:.3g} of its bound"


def check_forward(tl, x, w, b, eps=1e-5, xd=None):
    y64, m64, r64, xh = forward64(x, w, b, eps)
    xd = x.cuda() if xd is None else xd
    y, mean, rstd = tl.layer_norm(xd, w.cuda() if w is not None else None, b.cuda() if b is not None else None, eps)
    big = x.double().abs().amax(1)
    close("mean", mean, m64, 64 * U * big + 1e-30)
    # the variance is off by 64 u of itself (squares about the mean), and by the mean's error squared
    close("rstd", rstd, r64, 64 * U * r64 * (1 + (U * big * r64) ** 2))
    wa = w.double().abs() if w is not None else torch.ones(x.shape[1], dtype=torch.float64)
    ba = b.double().abs() if b is not None else torch.zeros(x.shape[1], dtype=torch.float64)
    into = (xh.abs() + (big * r64)[:, None]) * wa + ba
    close("y", y, y64, 64 * U * into + V[x.dtype] * y64.abs() + (2.0 ** -24 if x.dtype == torch.float16 else 1e-30))
    return y, mean, rstd


def check_backward(tl, dy, x, mean, rstd, w, dyd=None, xd=None):
    """mean, rstd: as the forward gave them, so that only the backward is judged."""
    dx64, dw64, db64, xh, g = backward64(dy, x, mean.cpu(), rstd.cpu(), w)
    dx, dw, db = tl.layer_norm_backward(dy.cuda() if dyd is None else dyd, x.cuda() if xd is None else xd, mean, rstd,
                                        w.cuda() if w is not None else None)
    r = rstd.cpu().double()[:, None]
    # xh is itself off by 4 u of x r and mean r, and the two means by 64 u of their terms' magnitudes
    xa = xh.abs() + (x.double().abs() + mean.cpu().double().abs()[:, None]) * r
    into = r * (g.abs() + g.abs().amax(1, keepdim=True) + xa * (g.abs() * xa).amax(1, keepdim=True))
    close("dx", dx, dx64, 64 * U * into + V[x.dtype] * dx64.abs() + (2.0 ** -24 if x.dtype == torch.float16 else 1e-30))
    rows = x.shape[0]
    close("dweight", dw, dw64, (rows + 64) * U * (dy.double().abs() * xa).sum(0) + 1e-30)
    close("dbias", db, db64, (rows + 64) * U * dy.double().abs().sum(0) + 1e-30)
    return dx, dw, db


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm(tl, rows, cols, dtype):
    x, dy, w, b = make(rows, cols, dtype, rows * 7 + cols)
    _, mean, rstd = check_forward(tl, x, w, b)
    check_backward(tl, dy, x, mean, rstd, w)


@pytest.mark.parametrize("pdtype", DTYPES)
@pytest.mark.parametrize("cols", [96, 2056])
def test_norm_parameter_types_and_none(tl, cols, pdtype):
    x, dy, w, b = make(11, cols, torch.bfloat16, 3, pdtype)
    for ww, bb in ((w, b), (w, None), (None, b), (None, None)):
        _, mean, rstd = check_forward(tl, x, ww, bb)
        check_backward(tl, dy, x, mean, rstd, ww)


@pytest.mark.parametrize("rows,cols", [(5000, 48), (4099, 1536), (1300, 4104), (700, 20000)])
def test_norm_many_rows(tl, rows, cols):
    """More rows than the grid holds: every CTA walks over several."""
    x, dy, w, b = make(rows, cols, torch.bfloat16, 5)
    _, mean, rstd = check_forward(tl, x, w, b)
    check_backward(tl, dy, x, mean, rstd, w)


@pytest.mark.parametrize("cols,ld,off", [(512, 520, 0), (512, 513, 0), (2048, 2056, 8), (2048, 2055, 1), (9000, 9004, 4)])
def test_norm_strided_rows(tl, cols, ld, off):
    """Row strides and starts on and off the 16-byte boundaries; what lies between the rows stays."""
    x, dy, w, b = make(9, cols, torch.bfloat16, 6)
    xb, db = (torch.full((9, ld), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    xd = torch.as_strided(xb, (9, cols), (ld, 1), off) if off + cols <= ld else None
    if xd is None:
        pytest.skip("the row does not fit")
    dyd = torch.as_strided(db, (9, cols), (ld, 1), off)
    xd.copy_(x)
    dyd.copy_(dy)
    _, mean, rstd = check_forward(tl, x, w, b, xd=xd)
    check_backward(tl, dy, x, mean, rstd, w, dyd=dyd, xd=xd)


def test_norm_large_mean(tl):
    """A mean 1000 times the deviation: the variance must not cancel."""
    x, dy, w, b = make(8, 4096, torch.float32, 8, mean=1000.0, scale=1.0)
    _, mean, rstd = check_forward(tl, x, w, b)
    check_backward(tl, dy, x, mean, rstd, w)


def test_norm_constant_row_and_one_column(tl):
    """No variance: y = b and rstd = 1 / sqrt(eps)."""
    x = torch.full((2, 640), 3.0).bfloat16().cuda()
    w, b = torch.full((640,), 2.0).bfloat16().cuda(), torch.full((640,), 0.5).bfloat16().cuda()
    y, mean, rstd = tl.layer_norm(x, w, b, 1e-4)
    assert torch.equal(y, torch.full_like(y, 0.5)) and torch.equal(mean.cpu(), torch.full((2,), 3.0))
    assert torch.allclose(rstd.cpu(), torch.full((2,), 100.0), rtol=1e-6)


@pytest.mark.parametrize("cols", [300, 3000, 30000])
def test_norm_nan_and_inf_stay_in_their_rows(tl, cols):
    x, dy, w, b = make(6, cols, torch.float32, 9)
    x[1, cols // 2] = float("nan")
    x[3, cols - 1] = float("inf")
    x[5, 0] = float("-inf")
    good = [0, 2, 4]
    y, mean, rstd = tl.layer_norm(x.cuda(), w.cuda(), b.cuda())
    y64, m64, r64, _ = forward64(x[good], w, b, 1e-5)
    assert torch.isnan(y[1]).all() and torch.isnan(y[3]).all() and torch.isnan(y[5]).all()
    assert torch.isnan(mean[1]) and mean[3] == float("inf") and mean[5] == float("-inf")
    assert torch.allclose(y[good].double().cpu(), y64, rtol=1e-5, atol=1e-5)
    dx, _, _ = tl.layer_norm_backward(dy.cuda(), x.cuda(), mean, rstd, w.cuda())
    assert torch.isnan(dx[1]).all() and torch.isfinite(dx[good]).all()


@pytest.mark.parametrize("cols", [40, 1500])
def test_norm_gradients_against_differences(tl, cols):
    """dx, dweight and dbias against central differences of the forward in 64 bits."""
    x, dy, w, b = make(4, cols, torch.float32, 10)
    _, mean, rstd = tl.layer_norm(x.cuda(), w.cuda(), b.cuda())
    dx, dw, db = (t.double().cpu() for t in tl.layer_norm_backward(dy.cuda(), x.cuda(), mean, rstd, w.cuda()))
    h = 1e-5
    loss = lambda x, w, b: (forward64(x, w, b, 1e-5)[0] * dy.double()).sum().item()  # noqa: E731
    rng = np.random.default_rng(0)
    for _ in range(12):
        r, c = int(rng.integers(4)), int(rng.integers(cols))
        for t, got in ((0, dx[r, c]), (1, dw[c]), (2, db[c])):
            args = [x.double(), w.double(), b.double()]
            step = torch.zeros_like(args[t])
            step[(r, c) if t == 0 else c] = h
            hi, lo = list(args), list(args)
            hi[t], lo[t] = args[t] + step, args[t] - step
            ref = (loss(*hi) - loss(*lo)) / (2 * h)
            # the difference's own error: h^2 (third derivative) and rounding 2^-52 |loss| / h
            assert abs(got.item() - ref) <= 1e-4 * max(1.0, abs(ref))


def test_norm_in_place_and_same_bits(tl):
    """y into x and dx into dy, and the same bits in every run."""
    x, dy, w, b = make(700, 1544, torch.bfloat16, 11)
    xd, dyd, wd, bd = (t.cuda() for t in (x, dy, w, b))
    y, mean, rstd = tl.layer_norm(xd, wd, bd)
    a = tl.layer_norm_backward(dyd, xd, mean, rstd, wd)
    c = tl.layer_norm_backward(dyd, xd, mean, rstd, wd)
    assert all(torch.equal(p, q) for p, q in zip(a, c))
    s = torch.cuda.current_stream().cuda_stream
    x2, dy2 = xd.clone(), dyd.clone()
    m2, r2 = torch.empty_like(mean), torch.empty_like(rstd)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    tl.tiled_linear_norm_forward(700, 1544, tl.TL_TYPE_BF16, x2.data_ptr(), 1544, tl.TL_TYPE_BF16, wd.data_ptr(),
                                 bd.data_ptr(), 1e-5, x2.data_ptr(), 1544, m2.data_ptr(), r2.data_ptr(), err.data_ptr(), s)
    assert torch.equal(x2, y)
    need = tl.tiled_linear_norm_backward_workspace_bytes(700, 1544)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    tl.tiled_linear_norm_backward(700, 1544, tl.TL_TYPE_BF16, dy2.data_ptr(), 1544, xd.data_ptr(), 1544,
                                  mean.data_ptr(), rstd.data_ptr(), tl.TL_TYPE_BF16, wd.data_ptr(), dy2.data_ptr(),
                                  1544, None, None, ws.data_ptr(), need, err.data_ptr(), s)
    assert torch.equal(dy2, a[0]) and not err.any()
    tl.check_operators()


def test_norm_no_rows(tl):
    x = torch.empty(0, 200, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = tl.layer_norm(x)
    assert y.shape == (0, 200) and mean.shape == (0,)
    dx, dw, db = tl.layer_norm_backward(x, x, mean, rstd)
    assert dx.shape == (0, 200) and not dw.any() and not db.any()


def test_norm_on_another_stream(tl):
    x, dy, w, b = make(256, 4096, torch.bfloat16, 12)
    s = torch.cuda.Stream()
    xd, wd, bd = x.cuda(), w.cuda(), b.cuda()
    want = tl.layer_norm(xd, wd, bd)[0]
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        x2 = xd * 1
        got = tl.layer_norm(x2, wd, bd)[0]
    s.synchronize()
    assert torch.equal(got, want)


def test_norm_offsets_past_32_bits(tl):
    """More than 2^31 elements: the last rows are where they belong."""
    rows, cols = 36000, 65536
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_()
    w, b = torch.ones(cols, device="cuda"), torch.zeros(cols, device="cuda")
    y, mean, rstd = tl.layer_norm(x, w, b)
    last = x[-3:].cpu()
    y64, m64, r64, _ = forward64(last, w.cpu(), b.cpu(), 1e-5)
    assert torch.allclose(mean[-3:].double().cpu(), m64, atol=1e-6) and torch.allclose(rstd[-3:].double().cpu(), r64, rtol=1e-5)
    assert torch.allclose(y[-3:].double().cpu(), y64, rtol=2.0 ** -8, atol=1e-5)
    dx, dw, db = tl.layer_norm_backward(x, x, mean, rstd, w)  # dy = x
    want = backward64(last, last, mean[-3:].cpu(), rstd[-3:].cpu(), w.cpu())[0]
    assert torch.allclose(dx[-3:].double().cpu(), want, rtol=2.0 ** -8, atol=1e-4)
    # dbias = column sums of x: 36000 terms of size one, fp32 (36000 u times their magnitudes, about 30000)
    assert torch.allclose(db[:64].double().cpu(), x[:, :64].double().sum(0).cpu(), atol=36000 * U * 30000)
