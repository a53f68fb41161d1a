"""The operators whose weight depends on the row, without a GPU: sizes whose work cannot be counted in 32 bits are invalid
arguments, refused like others before any CUDA call."""
import pytest

from test_row_operators_cpu import A, A_GOOD, AB, AB_GOOD, DW, DW_GOOD, DX, DX_GOOD, G, G_GOOD, refused, tl  # noqa: F401

M = 1 << 20


@pytest.mark.parametrize("kw", [
    # CTA pairs: 1024 groups of up to 2^21 blocks of rows by 2^8 of columns
    dict(R=1 << 29, K=8, n=1 << 16, groups=1024, ldx=8, x_rows=1 << 29, rows=None, ldw=1 << 16, w_apart=1 << 19, ldy=1 << 16),
    # single CTAs: 2^14 rows of 1024 groups (at most 1536 blocks of 32) by 2^21 of columns
    dict(R=1 << 14, K=8, n=1 << 28, groups=1024, ldx=8, x_rows=1 << 14, rows=None, ldw=1 << 28, w_apart=1 << 31, ldy=1 << 28)])
def test_too_many_tiles(tl, kw):  # noqa: F811
    refused(tl, tl.tiled_linear_grouped_forward, G, G_GOOD, kw, tl.TL_ERR_INVALID, "too many tiles")
    dx = dict(R=kw["R"], n=kw["K"], K=kw["n"], groups=kw["groups"], lddy=8, ldw=8, w_apart=kw["w_apart"], lddx=kw["n"])
    refused(tl, tl.tiled_linear_grouped_dx, DX, DX_GOOD, dx, tl.TL_ERR_INVALID, "too many tiles")


@pytest.mark.parametrize("kw", [
    # of 256 x 256: 2^16 by 2^16 of a matrix
    dict(R=8, K=1 << 24, n=1 << 24, groups=1, ldx=1 << 24, x_rows=8, rows=None, lddy=1 << 24, lddw=1 << 24, dw_apart=0),
    # of 128 by few columns: 2^23 of each of 1024 matrices
    dict(R=8, K=(1 << 30) - 8, n=8, groups=1024, ldx=1 << 30, x_rows=8, rows=None, lddy=8, lddw=8, dw_apart=1 << 33)])
def test_too_many_gradients(tl, kw):  # noqa: F811
    refused(tl, tl.tiled_linear_grouped_dw, DW, DW_GOOD, kw, tl.TL_ERR_INVALID, "too many tiles")


def test_too_many_adapter_tiles(tl):  # noqa: F811
    """2^29 rows by 2^30 columns: 2^22 blocks of rows by 2^23 of columns, eight of which a CTA takes."""
    n = (1 << 30) - 8
    wide = dict(T=1 << 29, n=n, r=8, adapters=2, ldb=1 << 30, b_apart=1 << 33, ldbase=1 << 30, bytes=1 << 60)
    refused(tl, tl.tiled_linear_adapter_forward, A, A_GOOD, dict(wide, ldy=1 << 30), tl.TL_ERR_INVALID, "too many tiles")
    wide = dict(T=1 << 29, K=n, r=8, adapters=2, ldx=1 << 30, a_apart=1 << 33, ldbase=1 << 30, lddx=1 << 30, da_apart=1 << 33, bytes=1 << 60)
    refused(tl, tl.tiled_linear_adapter_backward, AB, AB_GOOD, wide, tl.TL_ERR_INVALID, "too many tiles")


def test_base_under_the_result(tl):  # noqa: F811
    """The result may lie where base does only where each element of the one is that of the other."""
    for kw in (dict(base_type=2), dict(ldbase=72), dict(T=1, base_type=2)):
        refused(tl, tl.tiled_linear_adapter_forward, A, A_GOOD, kw, tl.TL_ERR_INVALID, "base")
        refused(tl, tl.tiled_linear_adapter_backward, AB, AB_GOOD, kw, tl.TL_ERR_INVALID, "base")
