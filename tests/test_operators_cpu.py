"""The operators around the product without a GPU: their entry points refuse bad
arguments before any CUDA call, with a status and a message, and size their
workspaces as the header says."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def tl():
    from offload_streamed_gb300 import _build
    _build.build()
    from offload_streamed_gb300 import tiled_linear
    tiled_linear.load()
    return tiled_linear


def refused(tl, fn, args, status, words):
    with pytest.raises(tl.TiledLinearError) as e:
        fn(*args)
    assert e.value.status == status, e.value
    assert words in str(e.value), e.value


def changed(names, good, **kw):
    return [kw.get(n, v) for n, v in zip(names, good)]


NF = ["rows", "cols", "type", "x", "ldx", "ptype", "w", "b", "eps", "y", "ldy", "mean", "rstd", "err", "stream"]
NF_GOOD = [4, 64, 0, 256, 64, 0, 256, 256, 1e-5, 256, 64, 256, 256, 256, None]
NB = ["rows", "cols", "type", "dy", "lddy", "x", "ldx", "mean", "rstd", "ptype", "w", "dx", "lddx", "dw", "db", "ws",
      "bytes", "err", "stream"]
NB_GOOD = [4, 64, 0, 256, 64, 256, 64, 256, 256, 0, 256, 256, 64, 256, 256, 256, 1 << 30, 256, None]


@pytest.mark.parametrize("kw,words", [
    (dict(rows=-1), "rows"), (dict(cols=0), "cols"), (dict(cols=131073, ldx=1 << 20, ldy=1 << 20), "131072"),
    (dict(type=3), "tl_type"), (dict(ptype=-1), "tl_type"), (dict(x=None), "null"), (dict(mean=None), "null"),
    (dict(x=257), "aligned"), (dict(rstd=258), "aligned"), (dict(w=257), "aligned"), (dict(ldx=63), "leading"),
    (dict(ldy=10), "leading"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(err=None), "err"),
    (dict(type=2, x=258), "aligned")])
def test_norm_forward_refusals(tl, kw, words):
    refused(tl, tl.tiled_linear_norm_forward, changed(NF, NF_GOOD, **kw), tl.TL_ERR_INVALID, words)


@pytest.mark.parametrize("kw,status,words", [
    (dict(dy=None), 1, "null"), (dict(lddy=1), 1, "leading"), (dict(dw=258), 1, "fp32"), (dict(dx=257), 1, "aligned"),
    (dict(ws=None), 3, "workspace"), (dict(ws=264), 3, "workspace"), (dict(bytes=4 * 2 * 64 * 4 - 1), 3, "workspace")])
def test_norm_backward_refusals(tl, kw, status, words):
    refused(tl, tl.tiled_linear_norm_backward, changed(NB, NB_GOOD, **kw), status, words)


def test_norm_workspace(tl):
    f = tl.tiled_linear_norm_backward_workspace_bytes
    assert f(4, 64) == 4 * 2 * 64 * 4        # a partial sum for each row at most
    assert f(1 << 20, 64) == 608 * 2 * 64 * 4
    assert f(1 << 20, 65536) == 76 * 2 * 65536 * 4
    assert f(-1, 64) == f(4, 0) == f(4, 131073) == 0 and f(0, 64) > 0


Q = ["rows", "cols", "type", "x", "ldx", "format", "rq", "ldr", "rs", "cq", "ldc", "cs", "tq", "ldt", "ts", "stream"]
Q_GOOD = [4, 64, 0, 256, 64, 0, 256, 64, 256, 256, 64, 256, 256, 64, 256, None]


@pytest.mark.parametrize("kw,words", [
    (dict(rows=-1), "rows"), (dict(cols=0), "cols"), (dict(type=9), "tl_type"), (dict(format=2), "tl_fp8_format"),
    (dict(rq=None, cq=None, tq=None), "no form"), (dict(x=None), "x is null"), (dict(x=257), "aligned"),
    (dict(ldx=63), "leading"), (dict(rs=None), "no scales"), (dict(ldc=63), "leading"), (dict(rs=258), "4-byte")])
def test_quantize_refusals(tl, kw, words):
    refused(tl, tl.tiled_linear_fp8_quantize, changed(Q, Q_GOOD, **kw), tl.TL_ERR_INVALID, words)


G = ["T", "K", "n", "fx", "x", "ldx", "xs", "fw", "w", "ldw", "ws", "y", "ldy", "err", "stream"]
G_GOOD = [4, 64, 64, 0, 256, 64, 256, 0, 256, 64, 256, 256, 64, 256, None]


@pytest.mark.parametrize("name", ["tiled_linear_fp8_gemm_forward", "tiled_linear_fp8_gemm_dx", "tiled_linear_fp8_gemm_dw"])
@pytest.mark.parametrize("kw,words", [
    (dict(T=-1), "T must"), (dict(K=0), "T must"), (dict(n=0), "T must"), (dict(K=1 << 31), "too large"),
    (dict(x=None), "null"), (dict(ws=None), "null"), (dict(y=None), "null"), (dict(err=None), "null"),
    (dict(x=264), "16-byte"), (dict(y=264), "16-byte"), (dict(ldx=72), "multiples of 16"), (dict(ldy=68), "multiple of 8"),
    (dict(ldx=48), "smaller"), (dict(ldy=56), "smaller"), (dict(fw=2), "tl_fp8_format"), (dict(xs=258), "4-byte")])
def test_product_refusals(tl, name, kw, words):
    refused(tl, getattr(tl, name), changed(G, G_GOOD, **kw), tl.TL_ERR_INVALID, words)


L = ["T", "K", "n", "type", "x", "ldx", "fw", "w", "ldw", "ws", "y", "ldy", "work", "bytes", "err", "stream"]
L_GOOD = [4, 64, 64, 0, 256, 64, 0, 256, 64, 256, 256, 64, 256, 1 << 20, 256, None]


@pytest.mark.parametrize("kw,status,words", [
    (dict(T=-1), 1, "T must"), (dict(n=1 << 30), 1, "T must"), (dict(w=None), 1, "null"), (dict(x=None), 1, "x is null"),
    (dict(type=5), 1, "tl_type"), (dict(ldy=60), 1, "multiple of 8"), (dict(work=None), 3, "workspace"),
    (dict(work=272), 3, "workspace"), (dict(bytes=511), 3, "workspace")])
def test_layer_forward_refusals(tl, kw, status, words):
    refused(tl, tl.tiled_linear_fp8_linear, changed(L, L_GOOD, **kw), status, words)


LB = ["T", "K", "n", "type", "x", "ldx", "dy", "lddy", "fw", "w", "ldw", "ws", "dx", "lddx", "dw", "lddw", "work",
      "bytes", "err", "stream"]
LB_GOOD = [4, 64, 64, 0, 256, 64, 256, 64, 0, 256, 64, 256, 256, 64, 256, 64, 256, 1 << 20, 256, None]


@pytest.mark.parametrize("kw,status,words", [
    (dict(dx=None, dw=None), 1, "neither"), (dict(x=None), 1, "x is null"), (dict(ldx=63), 1, "x is null"),
    (dict(dy=None), 1, "x is null"), (dict(lddw=60), 1, "multiple of 8"), (dict(err=None), 1, "null"),
    (dict(bytes=1535), 3, "workspace")])
def test_layer_backward_refusals(tl, kw, status, words):
    refused(tl, tl.tiled_linear_fp8_linear_backward, changed(LB, LB_GOOD, **kw), status, words)


def test_layer_workspaces(tl):
    up = lambda v, a: -(-v // a) * a  # noqa: E731
    held = lambda r, c, along, n: up(r * up(c, 16), 256) + up(-(-along // 512) * n * 4, 256)  # noqa: E731
    for T, K, n in ((1, 64, 64), (300, 1000, 77), (8192, 8192, 4096)):
        assert tl.tiled_linear_fp8_linear_workspace_bytes(T, K, n) == held(T, K, K, T)
        assert tl.tiled_linear_fp8_linear_backward_workspace_bytes(T, K, n) == held(T, n, n, T) + held(T, n, T, n) + held(T, K, T, K)
    assert tl.tiled_linear_fp8_linear_workspace_bytes(1, 0, 4) == 0


O = ["batch", "rows", "cols", "type", "g", "ldg", "apart", "steps", "a", "b", "c", "eps", "scale", "out", "ldo", "oapart",
     "ws", "bytes", "err", "stream"]
O_GOOD = [2, 64, 64, 0, 256, 64, 4096, 5, 1.0, 1.0, 1.0, 1e-7, 1.0, 256, 64, 4096, 256, 1 << 30, 256, None]


@pytest.mark.parametrize("kw,status,words", [
    (dict(batch=-1), 1, "batch"), (dict(batch=65536), 1, "batch"), (dict(rows=0), 1, "rows"), (dict(cols=(1 << 20) + 1), 1, "rows"),
    (dict(steps=0), 1, "steps"), (dict(steps=101), 1, "steps"), (dict(type=3), 1, "tl_type"), (dict(eps=-1.0), 1, "eps"),
    (dict(g=None), 1, "null"), (dict(err=None), 1, "null"), (dict(g=257), 1, "aligned"), (dict(out=264), 1, "16-byte"),
    (dict(ldo=68), 1, "multiples of 8"), (dict(oapart=4088), 1, "overlap"), (dict(ldg=63), 1, "leading"),
    (dict(ws=None), 3, "workspace"), (dict(ws=384 + 16), 3, "workspace"), (dict(bytes=1024), 3, "workspace")])
def test_orthogonalize_refusals(tl, kw, status, words):
    refused(tl, tl.tiled_linear_orthogonalize, changed(O, O_GOOD, **kw), status, words)


def test_nothing_to_do_needs_no_gpu(tl):
    """No rows, tokens or matrices: accepted before any CUDA call."""
    tl.tiled_linear_norm_forward(*changed(NF, NF_GOOD, rows=0, x=None, y=None, mean=None, rstd=None))
    tl.tiled_linear_fp8_quantize(*changed(Q, Q_GOOD, rows=0, x=None))
    tl.tiled_linear_fp8_gemm_forward(*changed(G, G_GOOD, T=0, x=None))
    tl.tiled_linear_fp8_linear(*changed(L, L_GOOD, T=0, x=None, work=None))
    tl.tiled_linear_orthogonalize(*changed(O, O_GOOD, batch=0, g=None, ws=None))


def test_functions_refuse_host_tensors_and_types(tl):
    x = torch.zeros(4, 64)
    for fn in (lambda: tl.layer_norm(x), lambda: tl.fp8_quantize(x, "row"), lambda: tl.orthogonalize(x),
               lambda: tl.layer_norm_backward(x, x, x[:, 0], x[:, 0])):
        with pytest.raises(tl.TiledLinearError) as e:
            fn()
        assert e.value.status == tl.TL_ERR_INVALID and "CUDA" in str(e.value)


def test_struct_free_signatures(tl):
    """The binding declares every argument of the new entry points (a forgotten one would be passed as a C int)."""
    lib = tl.load()
    for name, n in (("tiled_linear_norm_forward", 15), ("tiled_linear_norm_backward", 19), ("tiled_linear_fp8_quantize", 16),
                    ("tiled_linear_fp8_gemm_forward", 15), ("tiled_linear_fp8_linear", 16),
                    ("tiled_linear_fp8_linear_backward", 20), ("tiled_linear_orthogonalize", 20)):
        assert len(getattr(lib, name).argtypes) == n, name
    assert lib.tiled_linear_orthogonalize.argtypes[8] is ctypes.c_float
