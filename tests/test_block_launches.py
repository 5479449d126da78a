"""Launches of the block norms' backward pass at the ends of its ranges,
recorded on the host."""
import shutil

import pytest
import torch

import _launches
from error_feedback_quant_amd import echo

pytestmark = [pytest.mark.skipif(torch.cuda.is_available(), reason="host-only: launches are recorded, not made"),
              pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")]


@pytest.fixture(scope="module")
def recorder(tmp_path_factory):
    return _launches.build(tmp_path_factory.mktemp("recorder"))


def check_dims(got):
    for name, grid, block in got:
        assert min(grid) >= 1 and min(block) >= 1, (name, grid, block)
        assert grid[0] * block[0] < 1 << 32 and grid[1] * block[1] < 1 << 32 and grid[1] < 1 << 16, (name, grid, block)
        assert grid[0] * grid[1] * block[0] < 1 << 32, (name, grid, block)


GATE_TOKENS = [1, 2, 3, 4, 5, 99, 100, 101, 8192, 1 << 40, (1 << 63) - 100, (1 << 63) - 2, (1 << 63) - 1]


@pytest.mark.parametrize("T", [0, 1, 2, 3, 4, 100])
@pytest.mark.parametrize("H", [64, 1024, 8192, 9000])
def test_gate_rows_of_any_length(recorder, T, H):
    """Each gate row's gradient has its launch, and no row that is not there,
    up to the largest gate_tokens the type holds: more than T means one row."""
    calls = [dict(T=T, H=H, gate_tokens=n, gate=True) for n in GATE_TOKENS]
    for n, (rc, got) in zip(GATE_TOKENS, _launches.backward_launches(recorder, calls)):
        assert rc == 0, n
        if T == 0:
            continue
        check_dims(got)
        rows = -(-T // n)
        if H > 8192:
            gate = [g for g in got if "norm_bwd_gate_kernel" in g[0]]
            assert len(gate) == 1 and gate[0][1][1] == rows, (n, got)
        else:
            join = [g for g in got if "norm_bwd_sum_kernel" in g[0]]
            assert len(join) == 1, (n, got)
            # two strips of weights, then gate rows that groups share (a gate for each token leaves none)
            if n >= T:
                assert join[0][1][1] == 2 + 1, (n, got)
            else:
                assert 2 <= join[0][1][1] <= 2 + rows, (n, got)


@pytest.mark.parametrize("H", [64, 8192, 8193, 9000, 20000])
def test_no_tokens_make_one_launch(recorder, H):
    """Without tokens only the sums' kernel runs (it writes the weights' zero gradients), without a workspace."""
    (rc, got), (rc_gate, got_gate), (rc_none, got_none) = _launches.backward_launches(
        recorder, [dict(T=0, H=H), dict(T=0, H=H, gate_tokens=7, gate=True), dict(T=0, H=H, dw=False)])
    assert rc == 0 and rc_gate == 0 and rc_none == 0
    for g in (got, got_gate):
        check_dims(g)
        assert len(g) == 1 and "sum_kernel" in g[0][0], g
    assert not got_none
    assert echo.echo_block_norm_backward_workspace_bytes(0, H) == 0
