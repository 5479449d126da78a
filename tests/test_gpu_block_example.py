"""The block operators together with the all-reduce, as examples/tp_block.py runs them."""
import importlib.util
import os

import pytest
import torch

from _helpers import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tp_block():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tp_block.py")
    spec = importlib.util.spec_from_file_location("tp_block", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("bits,bound", [(8, 0.06), (4, 0.3)])
@pytest.mark.parametrize("tokens,hidden,ffn", [(64, 512, 1024), (4, 1024, 2048)])
def test_tp_block(tp_block, tokens, hidden, ffn, bits, bound):
    """A normal value's step in 8 bits is about 4 / 127 of its deviation, an
    error of 0.9 % of it; a product of two such operands is off by 1.3 %, two
    layers by about 2 %, and the 8-bit all-reduce adds 0.8 %: 0.06 is twice
    that.  The 4-bit all-reduce adds 10 % for each of its two quantizations
    (a step of 5.2 / 15 deviations), about 14 % in all: 0.3 is twice that."""
    say("tp block", tokens, hidden, ffn, bits)
    err, grads = tp_block.main(tokens, hidden, ffn, bits)
    torch.cuda.synchronize()
    assert err < bound
    assert all(bool(torch.isfinite(v).all()) and float(v.float().abs().max()) > 0 for v in grads.values())
