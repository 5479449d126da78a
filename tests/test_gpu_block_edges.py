"""The block operators on the GPU at the ends of their ranges, and in forms
that take sizes of their own."""
import numpy as np
import pytest
import torch

import _block_ref as ref
from _helpers import DEV, say
from test_gpu_block_int8 import matrix, same_bits, untouched
from test_gpu_block_norm import Case, run_backward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def echo():
    from error_feedback_quant_amd import echo as e
    assert torch.cuda.is_available()
    return e


@pytest.mark.parametrize("T", [1, 2, 3, 4, 100])
@pytest.mark.parametrize("H", [64, 1024, 9000])
@pytest.mark.parametrize("gate", [1 << 62, (1 << 63) - 100, (1 << 63) - 1])
def test_one_gate_row_for_any_number_of_tokens(echo, T, H, gate):
    """A gate row for more tokens than there are is one gate row, bit for bit, to the largest number the type holds."""
    say("one gate row", T, H, gate)
    c = Case(T, H, gate=T, beta=0.5)
    want = run_backward(echo, c)
    h = torch.empty_like(c.x)
    echo.echo_block_norm(c.args(echo, h=h))
    c.gate_tokens = gate
    got = run_backward(echo, c)
    hg = torch.empty_like(c.x)
    echo.echo_block_norm(c.args(echo, h=hg))
    torch.cuda.synchronize()
    assert set(got) == {"dx", "dr", "dw_post", "dw_pre", "dgate"}
    for k, v in got.items():
        same_bits(v, want[k])
    same_bits(hg, h)


@pytest.mark.parametrize("H", [64, 8192, 8193, 20000])
def test_no_tokens_at_every_width(echo, H):
    """No tokens: the weights' gradients are zeros, whichever form the width takes."""
    say("no tokens", H)
    x = torch.empty(0, H, device=DEV)
    dw = torch.full((2, H), 7.0, device=DEV)
    ws = torch.empty(max(16, echo.echo_block_norm_backward_workspace_bytes(0, H)), dtype=torch.uint8, device=DEV)
    echo.echo_block_norm_backward(echo.make_norm_args(x, x), echo.make_norm_grads(
        dh=x, dr_out=x, dx=x, dr=x, dw_post=dw[0], dw_pre=dw[1], workspace=ws))
    torch.cuda.synchronize()
    assert not bool(dw.any())
