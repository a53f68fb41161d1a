"""The orthogonalised update (through the package's function, so through the C ABI)
against the iteration in 64 bits.

Tolerance, as a share of the result's norm, derived from the kernel's roundings:
 * the result to bf16: 2^-9 of each element at most, 2^-9 / sqrt(3) of the norm
   in the mean: 1.13e-3, taken whole, 2^-9 = 1.95e-3;
 * a step rounds X, E = X X^T - s and Q to fp16 (2^-12 of the largest element of
   each, at most); these enter the next iterate through at most |b + 2cs| + 2 |c| |E|
   and |Q|, together under 4 for singular values in 0..1.3: 4 * 3 * 2^-12 * 1/sqrt(3)
   a step in the mean, and the map's slope there is at most about one in
   magnitude, so that the last steps' errors stay: sqrt(steps) of it at most:
   5 steps, 3.8e-3;
 * while singular values are small the map's slope equals its ratio, and relative
   errors pass on unchanged.
Together 6e-3 of the norm; elements within 8 of these of the root mean square."""
import pytest
import torch

pytestmark = pytest.mark.gpu

ABC = (3.4445, -4.7750, 2.0315)
TOL = 6e-3


@pytest.fixture(scope="module")
def tl():
    import __graft_entry__ as g
    g.build()
    from offload_streamed_gb300 import tiled_linear
    yield tiled_linear
    tiled_linear.check_operators()


def reference(g, steps=5, abc=ABC, eps=1e-7):
    x = g.double()
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    a, b, c = abc
    for _ in range(steps):
        p = x @ x.mT
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.mT if tall else x


def make(batch, rows, cols, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(batch, rows, cols, generator=g) * torch.exp(0.3 * torch.randn(batch, 1, cols, generator=g))
    k = max(1, min(rows, cols) // 16)
    x += torch.randn(batch, rows, k, generator=g) @ torch.randn(batch, k, cols, generator=g) / k ** 0.5
    return (x * 1e-3).to(dtype)


def close(got, ref, tol=TOL):
    got = got.double().cpu()
    assert got.shape == ref.shape and torch.isfinite(got).all()
    for a, b in zip(got.reshape(-1, *got.shape[-2:]), ref.reshape(-1, *ref.shape[-2:])):
        rms = b.square().mean().sqrt()
        assert (a - b).norm() <= tol * b.norm(), f"{((a - b).norm() / b.norm()).item():.3g}"
        assert ((a - b).abs() <= 8 * tol * torch.maximum(rms, b.abs())).all()


# one element to several tiles; wide, tall, square; ragged in tiles, K-blocks and 16-byte vectors
SHAPES = [(1, 1, 1), (1, 1, 9), (1, 7, 1), (2, 3, 5), (1, 16, 64), (3, 64, 16), (4, 200, 520), (1, 129, 264), (1, 300, 257),
          (2, 256, 256), (1, 257, 1000), (1, 1000, 130), (1, 513, 514), (1, 640, 1536), (1, 1100, 900), (9, 40, 72)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("batch,rows,cols", SHAPES)
def test_orthogonalize(tl, batch, rows, cols, dtype):
    g = make(batch, rows, cols, rows * 3 + cols, dtype)
    close(tl.orthogonalize(g.cuda()), reference(g))


def test_one_matrix_fp16_and_scale(tl):
    g = make(1, 130, 70, 1, torch.float16)[0]
    close(tl.orthogonalize(g.cuda(), scale=0.25), 0.25 * reference(g))


@pytest.mark.parametrize("steps", [1, 2, 3, 8])
def test_steps(tl, steps):
    g = make(2, 96, 160, steps)
    close(tl.orthogonalize(g.cuda(), steps=steps), reference(g, steps))


def test_other_coefficients(tl):
    """The cubic iteration (c = 0), which converges to the orthogonal factor itself."""
    g = make(1, 64, 200, 5)[0]
    abc = (1.5, -0.5, 0.0)
    got = tl.orthogonalize(g.cuda(), steps=25, coefficients=abc)
    close(got, reference(g, 25, abc))
    p = got.double().cpu() @ got.double().cpu().T
    assert (p - torch.eye(64)).abs().max() < 0.05


def test_large(tl):
    """Several tiles for every CTA pair, both sides."""
    for rows, cols in ((2048, 5000), (4500, 1800)):
        g = make(2, rows, cols, rows, torch.bfloat16).cuda()
        close(tl.orthogonalize(g), reference(g).cpu())


def test_strides(tl):
    big = make(3, 100, 90, 7, torch.bfloat16).cuda()
    for view in (big[:, 3:80, 5:66], big[1:, :, 1:], big[:, ::2], big[:, :, :88]):
        close(tl.orthogonalize(view), reference(view).cpu())


def test_zero_nan_and_independence(tl):
    g = make(4, 70, 50, 3)
    want = tl.orthogonalize(g.cuda())
    g[1] = 0
    g[2, 5, 7] = float("nan")
    got = tl.orthogonalize(g.cuda())
    assert not got[1].any() and torch.isnan(got[2]).all()
    assert torch.equal(got[0], want[0]) and torch.equal(got[3], want[3])


def test_same_bits_stream_and_empty(tl):
    g = make(2, 300, 700, 4, torch.bfloat16).cuda()
    a = tl.orthogonalize(g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = tl.orthogonalize(g * 1)
    s.synchronize()
    assert torch.equal(a, b)
    assert tl.orthogonalize(g[:0]).shape == (0, 300, 700)


def test_singular_values_near_one(tl):
    g = make(1, 512, 1024, 6)[0]
    s = torch.linalg.svdvals(tl.orthogonalize(g.cuda()).double().cpu())
    assert s.max() < 1.3 and s.min() > 0.3
