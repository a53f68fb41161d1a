"""The bound of the 8-bit gradients, on the CPU: an emulation of the rounded layer keeps it, and gradients with a mistake
do not."""
import pytest
import torch

from fp8_gradient_bound import layer64, near


def held(x, dim):
    """x in e4m3 with a power-of-two scale for each 128 elements along dim."""
    out = torch.empty_like(x)
    for i in range(0, x.shape[dim], 128):
        blk = x.narrow(dim, i, min(128, x.shape[dim] - i))
        scale = 2.0 ** torch.ceil(torch.log2(blk.abs().amax(dim, keepdim=True) / 448))
        out.narrow(dim, i, blk.shape[dim]).copy_((blk / scale).to(torch.float8_e4m3fn).float() * scale)
    return out


@pytest.mark.parametrize("T,K,n", [(3, 256, 1024), (300, 512, 768), (200, 4224, 264)])
def test_the_bound_tells_right_from_wrong(T, K, n):
    g = torch.Generator().manual_seed(T)
    x, w, dy = (torch.randn(a, b, generator=g) * torch.exp(0.5 * torch.randn(1, b, generator=g)) for a, b in ((T, K), (K, n), (T, n)))
    refs = layer64(x, w, dy)
    got = layer64(held(x, 1), held(w, 0), dy)[0], layer64(x, held(w, 1), held(dy, 1))[1], layer64(held(x, 0), w, held(dy, 0))[2]
    for a, ref in zip(got, refs):
        assert near(a.bfloat16().double(), ref)
        for wrong in (a * 0, a / 2, -a, a * 1.1, a.roll(1, 0), a.roll(1, 1)):
            assert not near(wrong, ref)
    # a sum that lacks its last block, and one element of a block's scale off by a power of two
    assert not near(layer64(x, held(w, 1)[:, :-128], held(dy, 1)[:, :-128])[1], refs[1])
    twice = held(dy, 1)
    twice[:, :128] *= 2
    assert not near(layer64(x, w, twice)[1], refs[1])
