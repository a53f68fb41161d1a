"""Which device's error word ``check_operators`` reads, without a GPU (the words are host tensors here), and what the
operators' entries refuse before they turn to the device."""
import pytest
import torch


@pytest.fixture
def tl(monkeypatch):
    from offload_streamed_gb300 import tiled_linear as tl
    words = {i: (torch.zeros(4, dtype=torch.int32), 0) for i in (0, 1)}
    waits = []
    monkeypatch.setattr(tl, "_err_words", words)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "synchronize", lambda d=None: waits.append((d, int(words[d][0][0]))))
    tl.waits = waits
    return tl


@pytest.mark.parametrize("device", [None, "cuda", "cuda:1", torch.device("cuda"), torch.device("cuda", 1)])
def test_current_device(tl, device):
    tl._err_words[0][0][0] = 3
    tl.check_operators(device)
    tl._err_words[1][0][0] = 5
    with pytest.raises(tl.TiledLinearError) as e:
        tl.check_operators(device)
    assert e.value.status == tl.TL_ERR_TIMEOUT and "0x5" in str(e.value)
    tl.check_operators(device)
    assert tl._err_words[0][0][0] == 3


@pytest.mark.parametrize("device", ["cuda:0", torch.device("cuda", 0)])
def test_named_device(tl, device):
    tl._err_words[1][0][0] = 5
    tl.check_operators(device)
    tl._err_words[0][0][0] = 3
    with pytest.raises(tl.TiledLinearError) as e:
        tl.check_operators(device)
    assert "0x3" in str(e.value) and tl._err_words[1][0][0] == 5


def test_cleared_before_another_stream_goes_on(tl):
    """The word is zero on the device when the error is raised: a bit that a later call sets is not lost."""
    tl._err_words[1][0][0] = 5
    with pytest.raises(tl.TiledLinearError):
        tl.check_operators()
    assert tl.waits == [(1, 5), (1, 0)]


def test_the_librarys_word_is_refused_without_a_place_for_it():
    from offload_streamed_gb300 import _build
    _build.build()
    from offload_streamed_gb300 import tiled_linear as tl
    assert tl.load().tiled_linear_operator_error_word(None) == tl.TL_ERR_INVALID


@pytest.mark.parametrize("x,dx", [(257, 256), (257, None)])
def test_a_backward_that_is_refused_enqueues_nothing(x, dx):
    """An x that does not fit its type is refused before dx's part is begun (which fails here for want of a device)."""
    from offload_streamed_gb300 import _build
    _build.build()
    from offload_streamed_gb300 import tiled_linear as tl
    with pytest.raises(tl.TiledLinearError) as e:
        tl.tiled_linear_fp8_linear_backward(4, 64, 64, tl.TL_TYPE_BF16, x, 64, 256, 64, 0, 256, 64, 256, dx, 64, 256, 64,
                                            256, 1 << 20, 256, None)
    assert e.value.status == tl.TL_ERR_INVALID and "aligned" in str(e.value), e.value


@pytest.mark.parametrize("name", ["fp8_matmul", "fp8_matmul_dx"])
def test_products_refuse_what_is_no_matrix(name):
    from offload_streamed_gb300 import tiled_linear as tl
    w, none = torch.zeros(4, 4).to(torch.float8_e4m3fn), torch.zeros(1, 1, dtype=torch.uint8)
    for shape in ((), (4,), (1, 4, 4)):
        with pytest.raises(tl.TiledLinearError) as e:
            getattr(tl, name)((torch.zeros(shape).to(torch.float8_e4m3fn), none), (w, none))
        assert e.value.status == tl.TL_ERR_INVALID and "fit" in str(e.value)
