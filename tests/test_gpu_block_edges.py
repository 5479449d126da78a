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


def one_signed(c):
    """Incoming gradients signed so that each column's terms mostly add up:
    dh along n_r, dr_out along x and above what h's gradient adds to it."""
    f = c.plain()
    sign = lambda v: torch.from_numpy(np.where(v < 0, -1.0, 1.0)).to(DEV)  # noqa: E731
    c.dh.copy_((sign(f["n_r"]) * c.dh.abs().double()).to(c.dh.dtype))
    c.up.copy_((sign(ref.f64(c.x)) * (4 + c.up.abs().double())).to(c.up.dtype))


@pytest.mark.parametrize("T,H,gate", [(300001, 24, 0), (300001, 24, 300001), (70003, 24, 1000), (70003, 20, 7), (70003, 24, 2500),
                                      (30001, 600, 30001), (20001, 1500, 0), (20001, 2100, 3000), (9001, 4100, 9001)])
def test_sums_over_many_tokens(echo, T, H, gate):
    """Sums whose terms have one sign, so that a lost, doubled or unwritten
    partial sum shows: the bound takes each form's own longest chain (under
    300 additions: 147 tokens of a group at most, the groups of a block, and
    a sixteenth of up to 1024 blocks with 16 waves)."""
    say("sums over many tokens", T, H, gate)
    c = Case(T, H, gate=gate, beta=0.5)
    if gate:
        c.gate.abs_()
    one_signed(c)
    f = c.plain()
    got = run_backward(echo, c)
    want, mag = ref.norm_backward(f, ref.f64(c.x), ref.f64(c.dh), ref.f64(c.up), ref.f64(c.gate), gate or 1, True, c.rho64,
                                  c.beta64)
    for k in ("dw_post", "dw_pre") + (("dgate",) if gate else ()):
        tol = (ref.backward_eps(f, H) + 300 * ref.U) * mag[k]
        share = np.quantile(tol / np.abs(want[k]), 0.95)
        assert share < 5e-4, (k, share)                    # a block's part (a thousandth and more) lies well outside the bound
        off = np.abs(ref.f64(got[k]) - want[k])
        assert (off <= tol + ref.U * np.abs(want[k])).all(), (k, float((off / tol).max()))


@pytest.mark.parametrize("T,K", [(3, 1025), (40, 1500), (5, 2047), (9, 4095), (3, 4097), (5, 9001), (2, 16383), (3, 16385)])
@pytest.mark.parametrize("pad,off", [(0, 0), (3, 1)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_quantize_tokens_that_end_inside_a_chunk(echo, T, K, pad, off, dt):
    say("quantize tail", T, K, pad, off, dt)
    d = torch.bfloat16 if dt == "bf16" else torch.float32
    rng = np.random.default_rng(K)
    v = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32))
    v[0, K - 1], v[-1, 0] = -90.0, 70.0                    # a largest value in the last, partial chunk
    _, x = matrix(T, K, K + pad, d, v, off)
    qb, q = matrix(T, K, K + pad, torch.int8, None, off)
    sb, s = matrix(1, T, T, torch.float32, None, off)
    echo.echo_quantize_tokens(x, K + pad, echo.BF16 if dt == "bf16" else echo.F32, T, K, q, K + pad, s)
    torch.cuda.synchronize()
    wq, ws = ref.quantize_tokens(x.float().cpu().numpy())
    same_bits(q, torch.from_numpy(wq))
    same_bits(s[0], torch.from_numpy(ws))
    untouched(qb, q)
    untouched(sb, s)


@pytest.mark.parametrize("M", [1, 2, 3, 4])
@pytest.mark.parametrize("N,K", [(40, 4097), (130, 5000), (64, 6144), (33, 8191), (256, 8192), (17, 4104)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("pad,off", [(0, 0), (8, 0), (5, 1)])
def test_linear_of_few_long_tokens(echo, M, N, K, dt, pad, off):
    """One launch with two chunks a thread: the codes and the product bit for bit, without a workspace."""
    say("linear long", M, N, K, dt, pad, off)
    d = torch.bfloat16 if dt == "bf16" else torch.float32
    rng = np.random.default_rng(M * N + K)
    v = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32))
    v[0, K - 1] = 60.0
    if M > 2:
        v[1, K // 2] = float("inf")
    _, x = matrix(M, K, K + pad, d, v, off)
    wv = torch.from_numpy(rng.integers(-128, 128, (N, K), dtype=np.int64).astype(np.int8))
    _, w = matrix(N, K, K + pad, torch.int8, wv, off)
    sw = torch.from_numpy(rng.uniform(0.001, 0.1, N).astype(np.float32))
    b = torch.from_numpy(rng.standard_normal(N).astype(np.float32))
    assert echo.echo_linear_int8_workspace_bytes(M, N, K) == 0
    wq, wsc = ref.quantize_tokens(x.float().cpu().numpy())
    for ydt, kind, bias in ((torch.float32, echo.F32, None), (torch.bfloat16, echo.BF16, b)):
        yb, y = matrix(M, N, N + pad, ydt, None, off)
        echo.echo_linear_int8(x, K + pad, echo.BF16 if dt == "bf16" else echo.F32, w, K + pad, sw.to(DEV),
                              None if bias is None else bias.to(DEV), M, N, K, y, N + pad, kind, None)
        torch.cuda.synchronize()
        want = torch.from_numpy(ref.gemm_int8(wq, wsc, wv.numpy(), sw.numpy(), None if bias is None else bias.numpy()))
        same_bits(y, want.to(ydt))
        untouched(yb, y)


@pytest.mark.parametrize("H", [513, 1023, 1025, 2049, 3001, 4095, 4097, 5001, 6143, 8191, 8193, 16383])
@pytest.mark.parametrize("x,r,h", [("bf16", "bf16", "bf16"), ("bf16", "f32", "bf16"), ("f32", "bf16", "f32"), ("f32", "f32", "f32"),
                                   ("bf16", "f32", "f32"), ("f32", "f32", "bf16"), ("f32", "bf16", "bf16"), ("bf16", "bf16", "f32")])
def test_rows_that_end_inside_a_chunk(echo, H, x, r, h):
    """Each width's form, forward (also to 8 bits) and backward, with a last chunk that is not full."""
    say("norm tail", H, x, r, h)
    check_forward(echo, Case(9, H, x, r, "bf16", "i8", gate=4, pad=3, off=1))
    check_forward(echo, Case(9, H, x, r, "f32", h, gate=4, beta=0.5))
    check_backward(echo, Case(9, H, x, r, "f32", h, gate=4, beta=0.5, pad=3, off=1))
    check_backward(echo, Case(14, H, x, r, "bf16", h, post=False))


@pytest.mark.parametrize("H", [1024, 5001, 9000])
def test_backward_far_rows(echo, H):
    """Rows past 2^31 elements: the same bits as for rows next to one another."""
    T, ld = 40, (1 << 31) // 39 + 8
    say("backward far rows", H)
    g = torch.Generator(device=DEV).manual_seed(H)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    v = rnd(4, T, H).bfloat16()
    w_post, w_pre, gate = 1 + 0.2 * rnd(H), 1 + 0.2 * rnd(H), 0.5 + 0.3 * rnd(T, H)
    ws = torch.empty(echo.echo_block_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device=DEV)
    out = []
    for dist in (H, ld):
        x, r, dh, up = (matrix(T, H, dist, torch.bfloat16, t)[1] for t in v)
        dx, dr = (matrix(T, H, dist, torch.bfloat16, None)[1] for _ in range(2))
        dw = torch.full((2, H), 7.0, device=DEV)
        dg = torch.full((T, H), 7.0, device=DEV)
        a = echo.make_norm_args(x, r, w_post=w_post, w_pre=w_pre, gate=gate, gate_tokens=1)
        echo.echo_block_norm_backward(a, echo.make_norm_grads(dh=dh, dr_out=up, dx=dx, dr=dr, dw_post=dw[0], dw_pre=dw[1], dgate=dg,
                                                              workspace=ws))
        torch.cuda.synchronize()
        out.append([t.contiguous().cpu() for t in (dx, dr, dw, dg)])
        del x, r, dh, up, dx, dr
    for p, q in zip(*out):
        same_bits(p, q)


def test_no_columns_in_8_bits(echo):
    """A token of no elements has the codes and the scale that quantizing it gives."""
    say("norm without columns")
    x = torch.empty(5, 0, device=DEV)
    for wide in (0, 16):
        s, want = (torch.full((6,), 7.0, device=DEV) for _ in range(2))
        h = torch.empty(5, wide, dtype=torch.int8, device=DEV)
        echo.echo_block_norm(echo.make_norm_args(x, h=h, h_scale=s[:5]))
        echo.echo_quantize_tokens(x, 0, echo.F32, 5, 0, h, wide, want[:5])
        torch.cuda.synchronize()
        assert float(want[0]) != 7.0
        same_bits(s, want)
