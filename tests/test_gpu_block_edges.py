"""The block operators on the GPU at the ends of their ranges, and in forms
that take sizes of their own."""
import numpy as np
import pytest
import torch

import _block_ref as ref
from _helpers import DEV, say
from test_gpu_block_int8 import matrix, same_bits, untouched
from test_gpu_block_norm import Case, check_backward, check_forward, run_backward

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
    bound = c.args

    def args(echo, **kw):                      # the number as it is, past the binding
        a = bound(echo, **kw)
        a.gate_tokens = gate
        return a
    c.args = args
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


WIDTHS = [64, 250, 1001, 2048, 4095, 4096, 8191, 8192, 16380, 16384, 17000]


def enlarge(c, rows_x, rows_r, factor):
    """Rows of x and of r times a factor that takes their squares out of fp32."""
    c.x[rows_x] = (c.x[rows_x].float() * factor).to(c.x.dtype)
    if c.r is not None:
        c.r[rows_r] = (c.r[rows_r].float() * factor).to(c.r.dtype)


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("h", ["f32", "bf16", "i8"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("factor", [1e18, 1e20, 2e37])
def test_norms_of_values_whose_squares_leave_fp32(echo, H, h, post, factor):
    """Rows of x, of r and of both up to 2e38 (squares to 4e76) between ordinary ones, by the formulas and their bounds."""
    say("norm large", H, h, post, factor)
    c = Case(7, H, x="f32" if H % 2 else "bf16", r="f32", h=h, post=post, gate=3, rho=0.9, beta=0.5)
    clean = check_forward(echo, c)
    enlarge(c, [1, 3, 6], [2, 3, 6], factor)
    assert bool(torch.isfinite(c.x).all()) and bool(torch.isfinite(c.r).all())
    got = check_forward(echo, c)
    keep = [0, 4, 5]
    for v, w in zip(got, clean):
        same_bits(v[keep].contiguous(), w[keep].contiguous())
    if h != "i8":
        assert bool((got[1][[1, 2, 3, 6]].float().abs().amax(1) > 0.5).all())      # no row has vanished


@pytest.mark.parametrize("H", WIDTHS)
@pytest.mark.parametrize("h", ["f32", "bf16", "i8"])
@pytest.mark.parametrize("bad", ["inf", "-inf", "nan"])
def test_norms_of_tokens_that_hold_no_number(echo, H, h, bad):
    """Every normed value of such a token is NaN, not only the one that stands
    where the infinity does; a residual sum has it there alone."""
    say("norm non-finite", H, h, bad)
    for post in (True, False):
        c = Case(6, H, x="f32", r="bf16", h=h, post=post)
        clean = check_forward(echo, c)
        c.x[1, H // 3] = float(bad)
        c.r[4, H - 1] = float(bad)
        r_out, h_out = c.out(c.kr)[1], c.out(c.kh)[1]
        s = torch.full((6,), 7.0, device=DEV)
        echo.echo_block_norm(c.args(echo, r_out=r_out, h=h_out, h_scale=s if h == "i8" else None))
        torch.cuda.synchronize()
        if h == "i8":
            assert not bool(h_out[[1, 4]].any()) and bool(torch.isnan(s[[1, 4]]).all())
        else:
            assert bool(torch.isnan(h_out[[1, 4]]).all())
        at = {1: H // 3, 4: H - 1}
        for t, k in at.items():
            off = ~torch.isfinite(r_out[t])
            if post and t == 1:
                assert bool(torch.isnan(r_out[t]).all())
            else:
                assert int(off.sum()) == 1 and bool(off[k])
                off[k] = False
                same_bits(r_out[t][torch.arange(H, device=DEV) != k], clean[0][t][torch.arange(H, device=DEV) != k])
        keep = [0, 2, 3, 5]
        for v, w in zip((r_out, h_out, s), clean):
            same_bits(v[keep].contiguous(), w[keep].contiguous())


LARGE_BWD = [(7, 64, 3), (9, 250, 0), (8, 1000, 1), (9, 1537, 4), (11, 2048, 0), (7, 4095, 100), (9, 4096, 2), (10, 5000, 3),
             (7, 8191, 0), (9, 8192, 7), (6, 9000, 4), (5, 17000, 0), (1000, 256, 3), (1000, 250, 64), (3000, 256, 601),
             (4000, 700, 1024), (2050, 300, 2049), (4100, 5000, 1024), (3000, 100, 0)]


@pytest.mark.parametrize("T,H,gate", LARGE_BWD)
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("factor", [1e15, 1e20, 1e30])
def test_gradients_of_values_whose_squares_leave_fp32(echo, T, H, gate, post, factor):
    """Such tokens among ordinary ones, in every form of the gate's sums: each
    gradient within its bound; without them no bit of the others' changes."""
    say("backward large", T, H, gate, post, factor)
    c = Case(T, H, x="bf16" if T % 2 else "f32", r="f32" if T % 2 else "bf16", w="f32", h="bf16" if T % 4 < 2 else "f32",
             post=post, gate=gate, rho=0.9, beta=0.5)
    clean = run_backward(echo, c)
    rng = np.random.default_rng(T + H)
    some = np.sort(rng.choice(T, max(2, T // 10), replace=False))
    rx, rr = some[::2].tolist(), (some[1::2] if T < 50 else some[1:]).tolist()
    enlarge(c, rx, rr, factor)
    got = check_backward(echo, c)
    keep = torch.from_numpy(np.setdiff1d(np.arange(T), some)).to(DEV)
    for k in ("dx", "dr"):
        same_bits(got[k][keep].contiguous(), clean[k][keep].contiguous())
    check_backward(echo, c, up=False)
    again = run_backward(echo, c, in_place=True)
    for k, v in again.items():
        same_bits(v, got[k])


@pytest.mark.parametrize("H", [64, 1000, 2048, 4096, 8192, 9000])
@pytest.mark.parametrize("bad", ["inf", "nan"])
def test_gradients_of_tokens_that_hold_no_number(echo, H, bad):
    """Gradients of such a token are NaN, those of the others keep their bits."""
    say("backward non-finite", H, bad)
    for post in (True, False):
        c = Case(9, H, x="f32", r="bf16", post=post, gate=2)
        clean = run_backward(echo, c)
        c.x[1, H // 3] = float(bad)
        c.r[4, H - 1] = float(bad)
        got = run_backward(echo, c)
        keep = [0, 2, 3, 5, 6, 7, 8]
        for k in ("dx", "dr"):
            same_bits(got[k][keep].contiguous(), clean[k][keep].contiguous())
            assert bool(torch.isnan(got[k][[1, 4]]).all())
        rows = [1, 3, 4]                      # gate rows without such a token
        same_bits(got["dgate"][rows].contiguous(), clean["dgate"][rows].contiguous())


@pytest.mark.parametrize("H", [64, 1000, 4096, 8192, 8200, 17000])
def test_sums_over_many_equal_tokens(echo, H):
    """60000 equal tokens behind one gate row: the sums are 60000 times one
    token's gradient.  A chain of T additions would be off by thousands of u
    (each addition rounds the same way for a while); the longest chain of any
    form is 235 tokens (60000 over 256 blocks or chunks) and 256 partial sums."""
    T = 60000
    say("equal tokens", H)
    one = Case(1, H, gate=1, beta=0.5)
    f = one.plain()
    want, mag = ref.norm_backward(f, ref.f64(one.x), ref.f64(one.dh), None, ref.f64(one.gate), 1, True, one.rho64, one.beta64)
    c = Case(1, H, gate=1, beta=0.5)
    c.T = c.gate_tokens = T
    for k in ("x", "r", "dh", "up"):
        setattr(c, k, getattr(one, k).repeat(T, 1))
    got = run_backward(echo, c, up=False, want=("dw_post", "dw_pre", "dgate"))
    for k in ("dw_post", "dw_pre", "dgate"):
        tol = (ref.backward_eps(f, H) + 500 * ref.U) * T * mag[k]
        assert float(np.median(tol / (T * np.abs(want[k]) + 1e-30))) < 2e-3, k       # the bound is a small part of the sum
        off = np.abs(ref.f64(got[k]) - T * want[k])
        assert (off <= tol + ref.U * T * np.abs(want[k])).all(), (k, float((off / tol).max()))
