"""The pre-norm layer example: the operators together, as a training loop and a
server would call them."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "prenorm_layer.py")


def test_layer_learns_and_serves():
    import __graft_entry__ as g
    g.build()
    from offload_streamed_gb300 import tiled_linear as tl
    spec = importlib.util.spec_from_file_location("prenorm_layer", PATH)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    layer = ex.train(tl, T=512, K=256, M=1024, N=4, steps=25)
    assert layer["losses"][-1] < 0.5 * layer["losses"][0]
    few, full = ex.answer(tl, layer, range(3)).float(), ex.streamed(tl, layer, 4)[:3].float()
    # two operands rounded to 4 bits: 2^-4 of each product at most, about 2^-4 / sqrt(3) in the mean, on both
    assert (few - full).norm() <= 2.0 ** -3 * full.norm()
