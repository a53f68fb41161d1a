"""The operators whose weight depends on the row without a GPU: their entry points refuse bad arguments before any CUDA
call, with a status and a message, and size their workspaces as the header says."""
import pytest
import torch


@pytest.fixture(scope="module")
def tl():
    from offload_streamed_gb300 import _build
    _build.build()
    from offload_streamed_gb300 import tiled_linear
    tiled_linear.load()
    return tiled_linear


def refused(tl, fn, names, good, kw, status, words):
    with pytest.raises(tl.TiledLinearError) as e:
        fn(*[kw.get(n, v) for n, v in zip(names, good)])
    assert e.value.status == status and words in str(e.value), e.value


GR = "T k groups ids slots rows offsets ws bytes stream".split()
GR_GOOD = [4, 2, 8, 256, 256, 256, 256, 256, 1 << 20, None]


@pytest.mark.parametrize("kw,status,words", [
    (dict(T=-1), 1, "tokens"), (dict(k=0), 1, "1..32"), (dict(k=33), 1, "1..32"), (dict(groups=0), 1, "1..1024"),
    (dict(groups=1025), 1, "1..1024"), (dict(T=1 << 30, k=2), 1, "too many"), (dict(ids=None), 1, "null"), (dict(offsets=None), 1, "offsets"),
    (dict(rows=258), 1, "aligned"), (dict(ws=None), 3, "workspace"), (dict(ws=384), 3, "workspace"), (dict(bytes=100), 3, "workspace")])
def test_group_rows_refusals(tl, kw, status, words):
    refused(tl, tl.tiled_linear_group_rows, GR, GR_GOOD, kw, status, words)


R = "T E k type logits ld normalize weights ids slots rows offsets ws bytes stream".split()
R_GOOD = [4, 8, 2, 0, 256, 8, 1, 256, 256, 256, 256, 256, 256, 1 << 20, None]


@pytest.mark.parametrize("kw,status,words", [
    (dict(k=9), 1, "experts"), (dict(type=3), 1, "tl_type"), (dict(logits=None), 1, "null"), (dict(weights=None), 1, "null"),
    (dict(logits=257), 1, "aligned"), (dict(type=2, logits=258), 1, "aligned"), (dict(ld=7), 1, "leading"), (dict(ids=None), 1, "null"),
    (dict(bytes=0), 3, "workspace")])
def test_route_refusals(tl, kw, status, words):
    refused(tl, tl.tiled_linear_route, R, R_GOOD, kw, status, words)


RB = "T E k type logits ld ids dweights normalize dlogits ldd stream".split()
RB_GOOD = [4, 8, 2, 0, 256, 8, 256, 256, 1, 256, 8, None]


@pytest.mark.parametrize("kw,words", [(dict(k=9), "experts"), (dict(type=-1), "tl_type"), (dict(dlogits=None), "null"), (dict(dweights=258), "aligned"),
                                      (dict(ldd=7), "leading"), (dict(T=-4), "tokens")])
def test_route_backward_refusals(tl, kw, words):
    refused(tl, tl.tiled_linear_route_backward, RB, RB_GOOD, kw, tl.TL_ERR_INVALID, words)


C = "T k cols rows type y ldy slots weights out ldout stream".split()
C_GOOD = [4, 2, 64, 8, 0, 256, 64, 256, 256, 256, 64, None]


@pytest.mark.parametrize("kw,words", [(dict(T=-1), "tokens"), (dict(k=33), "1..32"), (dict(cols=0), "cols"), (dict(cols=(1 << 20) + 1), "cols"),
                                      (dict(rows=-1), "rows"), (dict(type=4), "tl_type"), (dict(slots=None), "slots"), (dict(weights=258), "weights"),
                                      (dict(y=None), "y is null"), (dict(ldy=63), "y is null"), (dict(out=257), "out is null"), (dict(ldout=63), "out is null")])
def test_combine_refusals(tl, kw, words):
    refused(tl, tl.tiled_linear_combine, C, C_GOOD, kw, tl.TL_ERR_INVALID, words)


CB = "T k cols rows type dout lddout slots y ldy weights dy lddy dweights stream".split()
CB_GOOD = [4, 2, 64, 8, 0, 256, 64, 256, 256, 64, 256, 256, 64, 256, None]


@pytest.mark.parametrize("kw,words", [(dict(dout=None), "dout"), (dict(lddout=1), "dout"), (dict(dy=None), "dy"), (dict(y=None), "y is null"),
                                      (dict(dweights=258), "dweights"), (dict(slots=None), "slots")])
def test_combine_backward_refusals(tl, kw, words):
    refused(tl, tl.tiled_linear_combine_backward, CB, CB_GOOD, kw, tl.TL_ERR_INVALID, words)


G = "R K n groups type x ldx x_rows rows w ldw w_apart offsets y ldy ws bytes err stream".split()
G_GOOD = [4, 64, 64, 2, 0, 256, 64, 4, 256, 256, 64, 4096, 256, 256, 64, 256, 1 << 20, 256, None]


@pytest.mark.parametrize("kw,status,words", [
    (dict(R=-1), 1, "rows"), (dict(K=0), 1, "sizes"), (dict(n=1 << 31), 1, "sizes"), (dict(groups=1025), 1, "1..1024"), (dict(type=2), 1, "bf16"),
    (dict(x=None), 1, "null"), (dict(w=None), 1, "null"), (dict(y=None), 1, "null"), (dict(offsets=None), 1, "offsets"), (dict(err=None), 1, "err"),
    (dict(x=264), 1, "16-byte"), (dict(y=264), 1, "16-byte"), (dict(ldx=60), 1, "multiples of 8"), (dict(w_apart=4100), 1, "multiples of 8"),
    (dict(ldx=56), 1, "smaller"), (dict(ldw=56), 1, "smaller"), (dict(ldy=56), 1, "smaller"), (dict(w_apart=4088), 1, "overlap"),
    (dict(x_rows=0), 1, "too few"), (dict(rows=None, x_rows=3), 1, "too few"), (dict(rows=258), 1, "4-byte"), (dict(ldw=1 << 40), 1, "too large"),
    (dict(ws=None), 3, "workspace"), (dict(ws=128), 3, "workspace"), (dict(bytes=511), 3, "workspace")])
def test_grouped_refusals(tl, kw, status, words):
    if "ldw" in kw and kw["ldw"] > 1 << 30:
        kw = dict(kw, w_apart=1 << 50)
    refused(tl, tl.tiled_linear_grouped_forward, G, G_GOOD, kw, status, words)


DX = "R K n groups type dy lddy w ldw w_apart offsets dx lddx err stream".split()
DX_GOOD = [4, 64, 64, 2, 0, 256, 64, 256, 64, 4096, 256, 256, 64, 256, None]


@pytest.mark.parametrize("kw,words", [(dict(dy=None), "null"), (dict(dx=264), "16-byte"), (dict(lddx=56), "smaller"), (dict(type=5), "bf16")])
def test_grouped_dx_refusals(tl, kw, words):
    refused(tl, tl.tiled_linear_grouped_dx, DX, DX_GOOD, kw, tl.TL_ERR_INVALID, words)


DW = "R K n groups type x ldx x_rows rows dy lddy offsets dw lddw dw_apart ws bytes err stream".split()
DW_GOOD = [4, 64, 64, 2, 0, 256, 64, 4, 256, 256, 64, 256, 256, 64, 4096, 256, 1 << 20, 256, None]


@pytest.mark.parametrize("kw,status,words", [
    (dict(dw=None), 1, "dw is null"), (dict(lddw=60), 1, "multiples of 8"), (dict(lddw=56), 1, "smaller"), (dict(dw_apart=4088), 1, "smaller"),
    (dict(dy=None), 1, "null"), (dict(x=264), 1, "16-byte"), (dict(lddy=56), 1, "smaller"), (dict(x_rows=0), 1, "too few"),
    (dict(rows=None, x_rows=3), 1, "too few"), (dict(bytes=0), 3, "workspace")])
def test_grouped_dw_refusals(tl, kw, status, words):
    refused(tl, tl.tiled_linear_grouped_dw, DW, DW_GOOD, kw, status, words)


A = "T K n r adapters type x ldx a lda a_apart b ldb b_apart ids scale_dev scale base_type base ldbase y ldy h ldh ws bytes err stream".split()
A_GOOD = [4, 64, 64, 8, 2, 0, 256, 64, 256, 8, 512, 256, 64, 512, 256, 256, 1.0, 0, 256, 64, 256, 64, 256, 8, 256, 1 << 20, 256, None]


@pytest.mark.parametrize("kw,status,words", [
    (dict(T=-1), 1, "T must"), (dict(n=1 << 30), 1, "T must"), (dict(r=0), 1, "rank"), (dict(r=129), 1, "rank"), (dict(adapters=1025), 1, "adapters"),
    (dict(ids=None), 1, "ids"), (dict(ids=258), 1, "ids"), (dict(type=2), 1, "bf16"), (dict(x=None), 1, "null"), (dict(h=None, ldh=0), 1, "null"),
    (dict(y=None), 1, "null"), (dict(b=None), 1, "null"), (dict(b=264), 1, "16-byte"), (dict(y=264), 1, "16-byte"), (dict(ldy=56), 1, "leading"),
    (dict(ldb=60), 1, "multiples of 8"), (dict(ldb=56), 1, "smaller"), (dict(b_apart=504), 1, "overlap"), (dict(a_apart=504), 1, "overlap"),
    (dict(base_type=1), 1, "base"), (dict(base=257), 1, "base"), (dict(ldbase=63), 1, "base"), (dict(scale_dev=258), 1, "4-byte"),
    (dict(ws=None), 3, "workspace"), (dict(ws=264), 3, "workspace"), (dict(bytes=100), 3, "workspace")])
def test_adapter_refusals(tl, kw, status, words):
    refused(tl, tl.tiled_linear_adapter_forward, A, A_GOOD, kw, status, words)


AB = ("T K n r adapters type x ldx h ldh dy lddy a lda a_apart b ldb b_apart ids scale_dev scale base_type base ldbase dx lddx da ldda da_apart "
      "db lddb db_apart ws bytes err stream").split()
AB_GOOD = [4, 64, 64, 8, 2, 0, 256, 64, 256, 8, 256, 64, 256, 8, 512, 256, 64, 512, 256, 256, 1.0, 0, 256, 64, 256, 64, 256, 8, 512, 256, 64, 512,
           256, 1 << 20, 256, None]


@pytest.mark.parametrize("kw,status,words", [
    (dict(dx=None, da=None, db=None), 1, "null"), (dict(da=None), 1, "one of da and db"), (dict(db=None), 1, "one of da and db"),
    (dict(dy=None), 1, "null"), (dict(h=None), 1, "null"), (dict(ldh=4), 1, "multiples of 8"), (dict(dx=264), 1, "16-byte"),
    (dict(da_apart=504), 1, "smaller"), (dict(lddb=56), 1, "smaller"), (dict(ws=None), 3, "workspace")])
def test_adapter_backward_refusals(tl, kw, status, words):
    refused(tl, tl.tiled_linear_adapter_backward, AB, AB_GOOD, kw, status, words)


def test_workspaces(tl):
    assert tl.tiled_linear_route_workspace_bytes(10, 2, 64) == 65 * 152 * 4
    assert tl.tiled_linear_route_workspace_bytes(-1, 2, 64) == tl.tiled_linear_route_workspace_bytes(1, 33, 64) == 0
    assert tl.tiled_linear_grouped_workspace_bytes(100, 61) == 100 * 64 * 2
    assert tl.tiled_linear_grouped_workspace_bytes(0, 61) == 256 and tl.tiled_linear_grouped_workspace_bytes(5, 0) == 0
    up = lambda v: -(-v // 256) * 256  # noqa: E731
    T, r, n = 1000, 24, 5
    assert tl.tiled_linear_adapter_workspace_bytes(T, r, n) == 2 * up(T * 4) + up((n + 1) * 4) + up((n + 1) * 152 * 4) + up(T * 2 * 32 * 2)
    assert tl.tiled_linear_adapter_workspace_bytes(256, 16, 1) >= 256 * 16 * 16 * 4
    assert tl.tiled_linear_adapter_workspace_bytes(4, 129, 1) == tl.tiled_linear_adapter_workspace_bytes(4, 8, 0) == 0


def test_nothing_to_do_needs_no_gpu(tl):
    """No tokens or rows: accepted before any CUDA call (where nothing has to be written)."""
    call = lambda fn, names, good, **kw: fn(*[kw.get(n, v) for n, v in zip(names, good)])  # noqa: E731
    call(tl.tiled_linear_route_backward, RB, RB_GOOD, T=0, logits=None)
    call(tl.tiled_linear_combine, C, C_GOOD, T=0, y=None)
    call(tl.tiled_linear_combine_backward, CB, CB_GOOD, T=0, y=None)
    call(tl.tiled_linear_grouped_forward, G, G_GOOD, R=0, x=None, ws=None)
    call(tl.tiled_linear_grouped_dx, DX, DX_GOOD, R=0, dy=None)
    call(tl.tiled_linear_adapter_forward, A, A_GOOD, T=0, x=None, ws=None)


def test_functions_refuse(tl):
    x, ids = torch.zeros(4, 64), torch.zeros(4, 1, dtype=torch.int32)
    h = x.bfloat16()
    for fn, words in ((lambda: tl.route(x, 2), "CUDA"), (lambda: tl.group_rows(ids, 2), "CUDA"), (lambda: tl.combine(x, ids), "CUDA"),
                      (lambda: tl.combine_backward(x, ids), "CUDA"), (lambda: tl.route_backward(x, x, ids), "CUDA"),
                      (lambda: tl.grouped_linear(x, x, ids), "bfloat16"), (lambda: tl.grouped_linear(h, h, ids), "CUDA"),
                      (lambda: tl.adapter_linear(x, x, x, ids), "bfloat16"), (lambda: tl.adapter_linear(h, h, h, ids), "CUDA")):
        with pytest.raises(tl.TiledLinearError) as e:
            fn()
        assert e.value.status == tl.TL_ERR_INVALID and words in str(e.value), e.value


def test_signatures(tl):
    """The binding declares every argument (a forgotten one would be passed as a C int)."""
    lib = tl.load()
    for name, names in (("group_rows", GR), ("route", R), ("route_backward", RB), ("combine", C), ("combine_backward", CB), ("grouped_forward", G),
                        ("grouped_dx", DX), ("grouped_dw", DW), ("adapter_forward", A), ("adapter_backward", AB)):
        assert len(getattr(lib, "tiled_linear_" + name).argtypes) == len(names), name
