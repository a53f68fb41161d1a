"""Products grouped by expert through the C ABI, at the edges of their operands."""
import pytest
import torch

from rows_reference import check, grouped, grouped_backward
from test_gpu_grouped import normal, offsets_of, tl  # noqa: F401

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16
MARK = 0x5a5a


@pytest.mark.parametrize("tokens", [1, 7])
@pytest.mark.parametrize("K", [257, 1001, 1007])
def test_nothing_behind_a_row_is_read(tl, K, tokens):  # noqa: F811
    """Indexed rows of K elements, K no multiple of 8: what lies between them does not get into the workspace."""
    R, n, ld = 60, 264, (K + 7) // 8 * 8
    held = torch.full((tokens, ld), MARK, dtype=torch.int16, device="cuda").view(F16)
    held[:, :K] = normal(1, tokens, K, dtype=F16)
    x, w, dy = held[:, :K], normal(2, 2, K, n, dtype=F16), normal(3, R, n, dtype=F16)
    off, rows = offsets_of([40, 20]), (torch.arange(R, device="cuda") * 5 % tokens).int()
    y, dw = torch.empty(R, n, dtype=F16, device="cuda"), torch.empty(2, K, n, dtype=F16, device="cuda")
    need = tl.tiled_linear_grouped_workspace_bytes(R, K)
    works = [torch.zeros(need // 2, dtype=torch.int16, device="cuda") for _ in range(2)]
    err, stream = tl.tiled_linear_operator_error_word(), torch.cuda.current_stream().cuda_stream
    tl.tiled_linear_grouped_forward(R, K, n, 2, 1, x.data_ptr(), ld, tokens, rows.data_ptr(), w.data_ptr(), n, K * n, off.data_ptr(), y.data_ptr(), n,
                                    works[0].data_ptr(), need, err, stream)
    tl.tiled_linear_grouped_dw(R, K, n, 2, 1, x.data_ptr(), ld, tokens, rows.data_ptr(), dy.data_ptr(), n, off.data_ptr(), dw.data_ptr(), n, K * n,
                               works[1].data_ptr(), need, err, stream)
    check("y", y, *grouped(x, w, off, rows))
    check("dw", dw, *grouped_backward(x, dy, w, off, rows)[1])
    for work in works:
        assert work.any() and not (work == MARK).any()
    tl.check_operators()


def test_backward_refuses_before_it_begins(tl, monkeypatch):  # noqa: F811
    """What one of the backward's two products refuses is refused before the other is enqueued."""
    begun, real = [], tl.tiled_linear_grouped_dx
    monkeypatch.setattr(tl, "tiled_linear_grouped_dx", lambda *a: (begun.append(1), real(*a)))
    off, rows = offsets_of([3, 5]), torch.zeros(8, dtype=torch.int32, device="cuda")
    x, w, dy = normal(1, 4, 64), normal(2, 2, 64, 136), normal(3, 8, 136)
    with pytest.raises(tl.TiledLinearError) as e:
        tl.grouped_linear_backward(x[:0], dy, w, off, rows)
    assert e.value.status == tl.TL_ERR_INVALID and not begun
    tl.grouped_linear_backward(x, dy, w, off, rows)
    assert begun
