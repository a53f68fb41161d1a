"""Adapters in fp16 whose h, and whose dh in the backward, leave fp16's range or reach its subnormal numbers while the
results do not: against 64 bits, element by element, within bounds of an intermediate result that keeps its digits.

Two parts of a number whose place's largest lies in [2^14, 2^15): what the first rounds off is at most 2^-11 of it, and of
that the second again 2^-11, or half a subnormal step, 2^-25: 2^-22 of the number and 2^-39 of the place's largest.  In da
places of different sizes meet at the largest's unit, where either part may lose 2^-25 once more: 2^-39 twice, and once
for the place's own, of the largest of all: 3 * 2^-39."""
import pytest
import torch

import rows_reference
from rows_reference import adapter, adapter_backward, check
from test_gpu_adapter import both, case, normal, owners, tl  # noqa: F401

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def by_place(ref, before, dtype):
    size = ref.abs() + before
    return before + 2.0 ** -22 * size + 2.0 ** -39 * size.amax(1, keepdim=True)


def by_adapter(ref, before, dtype):
    size = ref.abs() + before
    return before + 2.0 ** -22 * size + 3 * 2.0 ** -39 * (size.max() if size.numel() else 0.0)


def checked(monkeypatch, names, got, refs, skip=()):
    """refs: () -> (value, bound) of each result, with the intermediate's error by place, or in da by adapter."""
    monkeypatch.setattr(rows_reference, "between", by_place)
    values = list(refs())
    if "da" in names:
        monkeypatch.setattr(rows_reference, "between", by_adapter)
        values[names.index("da")] = refs()[names.index("da")]
    for name, g, (ref, bound) in zip(names, got, values):
        if name not in skip:
            assert ref.abs().max() < 65504, f"{name} does not fit the type: {ref.abs().max()}"
            check(name, g, ref, bound)


def scaled(seed, size, *shape):
    """Normal values of a size given for all, or for each row."""
    return (normal(seed, *shape, dtype=F32) * size).to(F16)


# sizes of x, a, b for the forward, and of x, h, dy, a, b for the backward
SIZES = {"large": ((100.0, 60.0, 1e-3), (1e-3, 1e-2, 2000.0, 1e-3, 4.0)), "small": ((1e-2, 1e-4, 30.0), (100.0, 1.0, 1e-4, 30.0, 1e-3))}
SHAPES = [(256, 264, 392, 16, 5), (257, 264, 392, 16, 5), (40, 264, 392, 128, 3), (300, 200, 136, 24, 3), (700, 264, 392, 64, 2), (300, 72, 1030, 128, 4),
          (2000, 136, 264, 32, 1)]


@pytest.mark.parametrize("T,K,n,r,R", SHAPES)
@pytest.mark.parametrize("size", SIZES)
def test_forward(tl, monkeypatch, size, T, K, n, r, R):  # noqa: F811
    sx, sa, sb = SIZES[size][0]
    x, a, b = scaled(1, sx, T, K), scaled(2, sa, R, K, r), scaled(3, sb, R, r, n)
    ids, scale = owners(4, T, R, 3), torch.exp(0.3 * normal(5, R, dtype=F32))
    y, h = tl.adapter_linear(x, a, b, ids, scale=scale)
    # (h is returned in its own type: infinite where it leaves it)
    checked(monkeypatch, ("y", "h"), (y, h), lambda: adapter(x, a, b, ids, None, scale), skip=("h",) if size == "large" else ())
    if size == "large":
        assert torch.isinf(h).any()
    tl.check_operators()


@pytest.mark.parametrize("T,K,n,r,R", SHAPES)
@pytest.mark.parametrize("size", SIZES)
def test_backward(tl, monkeypatch, size, T, K, n, r, R):  # noqa: F811
    sx, sh, sg, sa, sb = SIZES[size][1]
    x, h, dy = scaled(1, sx, T, K), scaled(2, sh, T, r), scaled(3, sg, T, n)
    a, b, ids = scaled(4, sa, R, K, r), scaled(5, sb, R, r, n), owners(6, T, R, 3)
    dy[::3] = 0  # (rows that pass nothing back)
    scale = torch.exp(0.3 * normal(7, R, dtype=F32))
    got = tl.adapter_linear_backward(x, h, dy, a, b, ids, scale=scale)
    checked(monkeypatch, ("dx", "da", "db"), got, lambda: adapter_backward(x, h, dy, a, b, ids, None, scale))
    tl.check_operators()


@pytest.mark.parametrize("T", [200, 600, 3000])
def test_rows_of_different_sizes(tl, monkeypatch, T):  # noqa: F811
    """Six decades within an adapter: a place keeps its own digits in y and dx, and da those of its largest."""
    K, n, r, R = 264, 392, 16, 2
    g = torch.Generator(device="cuda").manual_seed(9)
    size = 10.0 ** (6 * torch.rand(T, 1, generator=g, device="cuda") - 4)
    x, a, b, ids = scaled(1, 10 * size, T, K), scaled(2, 1.0, R, K, r), scaled(3, 1e-2, R, r, n), owners(4, T, R, 3)
    y, h = tl.adapter_linear(x, a, b, ids)
    checked(monkeypatch, ("y", "h"), (y, h), lambda: adapter(x, a, b, ids, None, [1.0] * R))
    dy, x, h = scaled(5, size, T, n), scaled(6, 0.1, T, K), scaled(7, 0.1, T, r)
    got = tl.adapter_linear_backward(x, h, dy, a, b, ids, scale=0.25)
    checked(monkeypatch, ("dx", "da", "db"), got, lambda: adapter_backward(x, h, dy, a, b, ids, None, [0.25] * R))
    tl.check_operators()


@pytest.mark.parametrize("base", [None, F16, F32])
@pytest.mark.parametrize("r", [1, 8, 24, 32, 64, 100, 128])
@pytest.mark.parametrize("T", [20, 300])
def test_ranks(tl, monkeypatch, T, r, base):  # noqa: F811
    monkeypatch.setattr(rows_reference, "between", by_adapter)
    both(tl, *case(T, 264, 392, r, 5, F16), base_dtype=base)


def test_an_infinite_row_stays_one(tl):  # noqa: F811
    """A row of infinities changes no bit of the others' y and dx, and none of the other adapters' gradients."""
    T, K, n, r, R = 400, 136, 264, 16, 3
    x, a, b, ids, scale = case(T, K, n, r, R, F16)
    h, dy = normal(8, T, r, dtype=F16), normal(9, T, n, dtype=F16)
    good = *tl.adapter_linear(x, a, b, ids, scale=scale), *tl.adapter_linear_backward(x, h, dy, a, b, ids, scale=scale)
    row = (ids == 1).nonzero()[7, 0]
    x[row], dy[row] = float("inf"), float("inf")
    bad = *tl.adapter_linear(x, a, b, ids, scale=scale), *tl.adapter_linear_backward(x, h, dy, a, b, ids, scale=scale)
    keep = torch.arange(T, device="cuda") != row
    for i in (0, 1, 2):
        assert torch.equal(good[i][keep], bad[i][keep]) and not torch.isfinite(bad[i][row]).any(), i
    for i in (3, 4):
        assert torch.equal(good[i][[0, 2]], bad[i][[0, 2]]) and not torch.isfinite(bad[i][1]).all(), i


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("T", [20, 300])
def test_bf16_at_the_end_of_its_range(tl, T, sign):  # noqa: F811
    """h and dh finite in 32 bits, but past the largest bf16 by more than half a step: 2^127 (2 - 2^-7 + 1.5 2^-8)."""
    r = 16
    big, rest = 2.0 ** 64 * (2 - 2.0 ** -7), 2.0 ** 64 * 1.5 * 2.0 ** -8
    x = torch.full((T, 8), sign * 2.0 ** 63, device="cuda").to(BF16)
    a = torch.zeros(1, 8, r, device="cuda").to(BF16)
    a[:, 0], a[:, 1] = big, rest
    b = torch.full((1, r, 8), 2.0 ** -120, device="cuda").to(BF16)
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    ref = sign * 2.0 ** 63 * (big + rest) * r * 2.0 ** -120
    y, h = tl.adapter_linear(x, a, b, ids)
    assert ((y.double() - ref).abs() <= 2.0 ** -7 * abs(ref)).all() and torch.isinf(h).all()
    # the same as dh = dy . b^T, with the factors turned
    dx, da, db = tl.adapter_linear_backward((x[:, :2] * 2.0 ** -100).contiguous(), torch.zeros_like(h), x, b[:, :, :2].transpose(1, 2).contiguous(),
                                            a.transpose(1, 2).contiguous(), ids)
    assert ((dx.double() - ref).abs() <= 2.0 ** -7 * abs(ref)).all() and not db.any()


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_scales_of_adapters_without_rows(tl, dtype):  # noqa: F811
    """A sum of nothing is zero, whatever its adapter's scale."""
    for T in (20, 300):
        x, a, b, ids, _ = case(T, 72, 136, 16, 4, dtype)
        ids[ids == 2] = -1
        scale = torch.tensor([1.0, 0.5, float("inf"), 2.0], device="cuda")
        h, dy = normal(8, T, 16, dtype=dtype), normal(9, T, 136, dtype=dtype)
        good = tl.adapter_linear_backward(x, h, dy, a, b, ids, scale=scale.clamp(max=2.0))
        for bad in (float("inf"), float("nan")):
            scale[2] = bad
            got = tl.adapter_linear_backward(x, h, dy, a, b, ids, scale=scale)
            assert all(torch.equal(p, q) for p, q in zip(good, got)) and not got[1][2].any() and not got[2][2].any()


def test_same_bits_again_and_in_a_graph(tl):  # noqa: F811
    """Inputs of other sizes in a captured call: the units are found anew, and the bits are those of a call by itself."""
    T, K, n, r, R = 600, 264, 392, 32, 3
    _, a, b, _, scale = case(1, K, n, r, R, F16)
    inputs = []
    for s, size in enumerate((1.0, 300.0, 1e-4)):
        inputs.append((scaled(s, size, T, K), scaled(10 + s, size, T, n), scaled(20 + s, 1.0, T, r), owners(s, T, R, 5)))

    def call(x, dy, h, ids):
        return *tl.adapter_linear(x, a, b, ids, scale=scale), *tl.adapter_linear_backward(x, h, dy, a, b, ids, scale=scale)

    want = [call(*i) for i in inputs]
    held = [t.clone() for t in inputs[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(*held)
    for i in (1, 2, 0, 2, 1):
        for t, s in zip(held, inputs[i]):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want[i])), i
        assert all(torch.equal(p, q) for p, q in zip(call(*inputs[i]), want[i])), i
    tl.check_operators()
