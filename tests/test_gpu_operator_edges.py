"""Edges of the operators that their own files do not reach: results of norm in rows with gaps, the few-token product's
route for more than 128 tokens in the forward, the 8-bit gradients against the layer without rounding."""
import numpy as np
import pytest
import torch

import test_gpu_norm as norm
from fp8_gradient_bound import ROUNDING, layer64, near
from test_gpu_fp8 import compare, make, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tl():
    import __graft_entry__ as g
    g.build()
    from offload_streamed_gb300 import tiled_linear
    yield tiled_linear
    tiled_linear.check_operators()


class IntoGaps:
    """layer_norm and layer_norm_backward of tiled_linear, whose matrices lie in rows of `cols` + `gap` elements from
    element `off` of a buffer on: what is not theirs has to keep its bits."""

    def __init__(self, tl, gap, off):
        self.tl, self.gap, self.off = tl, gap, off

    def place(self, x):
        rows, cols = x.shape
        word = torch.int32 if x.dtype == torch.float32 else torch.int16
        buf = torch.full((self.off + rows * (cols + self.gap) + 64,), 0x5a5a, dtype=word, device="cuda")
        return buf, torch.as_strided(buf.view(x.dtype), (rows, cols), (cols + self.gap, 1), self.off)

    def checked(self, buf, view):
        left = buf.clone()
        torch.as_strided(left, view.shape, view.stride(), self.off).fill_(0x5a5a)
        assert (left == 0x5a5a).all(), "written outside the result"
        return view

    def layer_norm(self, x, w, b, eps):
        tl, (rows, cols) = self.tl, x.shape
        kind = norm.DTYPES.index(x.dtype)
        buf, y = self.place(x)
        mean, rstd = (torch.empty(rows, device="cuda") for _ in range(2))
        tl.tiled_linear_norm_forward(rows, cols, kind, x.data_ptr(), x.stride(0), kind, w.data_ptr(), b.data_ptr(), eps,
                                     y.data_ptr(), cols + self.gap, mean.data_ptr(), rstd.data_ptr(),
                                     tl.tiled_linear_operator_error_word(), torch.cuda.current_stream().cuda_stream)
        return self.checked(buf, y), mean, rstd

    def layer_norm_backward(self, dy, x, mean, rstd, w):
        tl, (rows, cols) = self.tl, x.shape
        kind = norm.DTYPES.index(x.dtype)
        buf, dx = self.place(x)
        dw, db = (torch.empty(cols, device="cuda") for _ in range(2))
        need = tl.tiled_linear_norm_backward_workspace_bytes(rows, cols)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        tl.tiled_linear_norm_backward(rows, cols, kind, dy.data_ptr(), dy.stride(0), x.data_ptr(), x.stride(0),
                                      mean.data_ptr(), rstd.data_ptr(), kind, w.data_ptr(), dx.data_ptr(), cols + self.gap,
                                      dw.data_ptr(), db.data_ptr(), ws.data_ptr(), need,
                                      tl.tiled_linear_operator_error_word(), torch.cuda.current_stream().cuda_stream)
        return self.checked(buf, dx), dw, db


@pytest.mark.parametrize("dtype", norm.DTYPES)
@pytest.mark.parametrize("gap,off", [(16, 0), (16, 8), (3, 0), (16, 1), (5, 3)])
@pytest.mark.parametrize("rows,cols", [(30, 256), (30, 250), (9, 2048), (700, 1544), (5, 9000)])
def test_norm_into_rows_with_gaps(tl, rows, cols, gap, off, dtype):
    """Rows of a warp, a CTA and a cluster: on 16-byte boundaries, with a stride or a start that is not, and columns
    that no vector divides."""
    x, dy, w, b = norm.make(rows, cols, dtype, rows + cols)
    into = IntoGaps(tl, gap, off)
    _, mean, rstd = norm.check_forward(into, x, w, b)
    norm.check_backward(into, dy, x, mean, rstd, w)


# more than 128 tokens, few output tiles, reductions of 32 blocks and more: whole and ragged in each
@pytest.mark.parametrize("T,K,n", [(129, 4096, 128), (256, 4100, 520), (300, 8192, 264), (1000, 5000, 72), (2100, 4224, 392)])
def test_forward_in_several_blocks_of_tokens(tl, T, K, n):
    x, w = make(T, K, 1, spread=1.0).cuda(), make(K, n, 2, spread=0.2).cuda()
    xq, wq = tl.fp8_quantize(x, "row"), tl.fp8_quantize(w, "tile")
    xv, wv = values(*xq, "row"), values(*wq, "tile")
    compare("y", tl.fp8_linear(x, *wq), xv, wv, K)
    compare("y of the forms", tl.fp8_matmul(xq, wq), xv, wv, K)


@pytest.mark.parametrize("T,K,n", [(3, 256, 1024), (300, 512, 768), (200, 4224, 264)])
def test_gradients_against_the_layer_without_rounding(tl, T, K, n):
    """All of dx and dw against the 64-bit gradient by the unrounded operands, and y against its product."""
    x, w, dy = make(T, K, 1, spread=0.0), make(K, n, 2, spread=0.0), make(T, n, 3, spread=0.0)
    wq, ws = tl.fp8_quantize(w.cuda(), "tile")
    got = (tl.fp8_linear(x.cuda(), wq, ws), *tl.fp8_linear_backward(x.cuda(), dy.cuda(), wq, ws))
    for name, a, ref in zip(("y", "dx", "dw"), got, layer64(x, w, dy)):
        assert near(a.double().cpu(), ref), f"{name}: {((a.double().cpu() - ref).norm() / ref.norm()).item():.3g} > {ROUNDING:.3g}"
