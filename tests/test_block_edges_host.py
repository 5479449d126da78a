"""The block operators' binding and definitions at the ends of their ranges, without a GPU."""
import ctypes

import pytest
import torch

from error_feedback_quant_amd import echo


@pytest.mark.parametrize("gate_tokens", [6, 7, (1 << 63) - 1, 1 << 63, 1 << 64, (1 << 64) + 1, 10 ** 30])
def test_binding_keeps_large_gate_tokens_whole(gate_tokens):
    """One gate row for all tokens, however large its number of tokens: the C
    side's 64 bits must not take another number from it."""
    x = torch.zeros(6, 32, dtype=torch.bfloat16)
    a = echo.make_norm_args(x, gate=torch.ones(1, 32), gate_tokens=gate_tokens)
    assert a.gate_tokens >= 6
    assert echo.make_norm_args(torch.zeros(0, 32), gate=torch.ones(0, 32), gate_tokens=gate_tokens).gate_tokens >= 1


def test_scales_without_columns_are_checked():
    """A norm to 8 bits of no elements still writes its scales, so their pointer is checked."""
    if torch.cuda.is_available():
        pytest.skip("host-only argument checks (a GPU is visible)")
    a = echo.NormArgs()
    a.T, a.H, a.h_dtype, a.eps, a.res_scale, a.block_scale = 3, 0, echo.I8, 1e-5, 1.0, 1.0
    a.h_scale = (1 << 20) + 2
    assert echo.lib().echo_block_norm(ctypes.byref(a), None) == echo.EALIGN
    a.h_scale = None
    assert echo.lib().echo_block_norm(ctypes.byref(a), None) == echo.OK
