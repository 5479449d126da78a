"""The block operators without a GPU: the host's refusals, the workspace
sizes, the binding's checks of tensors, and the plain 64-bit forms that the
GPU tests compare with (gradients against central differences)."""
import numpy as np
import pytest
import torch

import _block_ref as ref
from error_feedback_quant_amd import echo

FAKE = 1 << 20          # 16-byte aligned, never dereferenced: the calls below are refused or empty


@pytest.fixture
def host_only():
    if torch.cuda.is_available():
        pytest.skip("host-only argument checks (a GPU is visible)")


def rc_of(fn, *args, **kw):
    try:
        fn(*args, **kw)
        return 0
    except echo.EchoError as e:
        return e.rc


def test_quantize_tokens_refusals(host_only):
    def q(**kw):
        a = dict(x=FAKE, dt=echo.BF16, ldx=64, T=4, K=64, q=FAKE, ldq=64, s=FAKE) | kw
        return rc_of(echo.echo_quantize_tokens, a["x"], a["ldx"], a["dt"], a["T"], a["K"], a["q"], a["ldq"], a["s"], stream=0)
    assert q(dt=echo.I8) == echo.EUNSUP and q(dt=-1) == echo.EUNSUP
    assert q(T=-1) == echo.ESHAPE and q(K=-1) == echo.ESHAPE and q(T=1 << 31) == echo.ESHAPE
    assert q(K=131072, ldx=131072, ldq=131072) == echo.ESHAPE
    assert q(ldx=63) == echo.ESHAPE and q(ldq=63) == echo.ESHAPE and q(ldx=1 << 40) == echo.ESHAPE
    assert q(x=None) == echo.EINVAL and q(q=None) == echo.EINVAL and q(s=None) == echo.EINVAL
    assert q(x=FAKE + 1) == echo.EALIGN and q(s=FAKE + 2) == echo.EALIGN and q(x=FAKE + 2, dt=echo.F32) == echo.EALIGN
    assert q(T=0, x=None) == 0


def gemm(**kw):
    a = dict(x=FAKE, ldx=64, sx=FAKE, w=FAKE, ldw=64, sw=FAKE, bias=None, M=4, N=8, K=64, y=FAKE, ldy=8, dt=echo.BF16) | kw
    return rc_of(echo.echo_gemm_int8, a["x"], a["ldx"], a["sx"], a["w"], a["ldw"], a["sw"], a["bias"], a["M"], a["N"],
                 a["K"], a["y"], a["ldy"], a["dt"], stream=0)


def linear(**kw):
    a = dict(x=FAKE, xd=echo.BF16, ldx=64, w=FAKE, ldw=64, sw=FAKE, bias=None, M=300, N=8, K=64, y=FAKE, ldy=8,
             dt=echo.BF16, ws=FAKE, wb=1 << 30) | kw
    return rc_of(echo.echo_linear_int8, a["x"], a["ldx"], a["xd"], a["w"], a["ldw"], a["sw"], a["bias"], a["M"], a["N"],
                 a["K"], a["y"], a["ldy"], a["dt"], a["ws"], a["wb"], stream=0)


@pytest.mark.parametrize("fn", [gemm, linear])
def test_product_refusals(host_only, fn):
    assert fn(dt=echo.I8) == echo.EUNSUP and fn(dt=9) == echo.EUNSUP
    assert fn(M=-1) == echo.ESHAPE and fn(N=-1) == echo.ESHAPE and fn(K=-1) == echo.ESHAPE
    assert fn(K=131072, ldx=131072, ldw=131072) == echo.ESHAPE          # 2^14 * 2^17 passes 2^31 - 1
    assert fn(ldx=63) == echo.ESHAPE and fn(ldw=63) == echo.ESHAPE and fn(ldy=7) == echo.ESHAPE
    assert fn(M=(1 << 31) - 1, N=(1 << 31) - 1, ldy=1 << 31) == echo.ESHAPE
    assert fn(x=None) == echo.EINVAL and fn(w=None) == echo.EINVAL and fn(sw=None) == echo.EINVAL
    assert fn(y=None) == echo.EINVAL
    assert fn(sw=FAKE + 2) == echo.EALIGN and fn(bias=FAKE + 1) == echo.EALIGN
    assert fn(y=FAKE + 1) == echo.EALIGN and fn(y=FAKE + 2, dt=echo.F32) == echo.EALIGN
    assert fn(M=0, x=None, y=None) == 0 and fn(N=0, w=None, y=None) == 0


def test_product_refusals_of_their_own(host_only):
    assert gemm(sx=None) == echo.EINVAL and gemm(sx=FAKE + 2) == echo.EALIGN
    assert linear(xd=echo.I8) == echo.EUNSUP and linear(x=FAKE + 1) == echo.EALIGN
    need = echo.echo_linear_int8_workspace_bytes(300, 8, 64)
    assert need == 300 * 64 + 300 * 4
    assert linear(ws=None) == echo.EINVAL and linear(wb=need - 1) == echo.EINVAL and linear(ws=FAKE + 4) == echo.EALIGN
    assert echo.echo_linear_int8_workspace_bytes(300, 8, 131072) == 0
    assert echo.echo_linear_int8_workspace_bytes(-1, 8, 64) == 0


def norm_args(**kw):
    a = echo.NormArgs()
    a.T, a.H = 4, 64
    a.ld_x = a.ld_r = a.ld_r_out = a.ld_h = a.ld_gate = 64
    a.gate_tokens = 0
    a.x_dtype = a.r_dtype = a.w_dtype = a.h_dtype = echo.BF16
    a.post, a.eps, a.res_scale, a.block_scale = 1, 1e-5, 1.0, 1.0
    a.x = a.r = a.r_out = a.h = FAKE
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_block_norm_refusals(host_only):
    f = lambda **kw: rc_of(echo.echo_block_norm, norm_args(**kw), stream=0)  # noqa: E731
    for k in ("x_dtype", "r_dtype", "w_dtype"):
        assert f(**{k: echo.I8}) == echo.EUNSUP and f(**{k: 5}) == echo.EUNSUP
    assert f(h_dtype=3) == echo.EUNSUP
    assert f(T=-1) == echo.ESHAPE and f(H=-1) == echo.ESHAPE and f(T=1 << 31) == echo.ESHAPE
    assert f(H=(1 << 30) + 1) == echo.ESHAPE
    for k in ("ld_x", "ld_r", "ld_r_out", "ld_h"):
        assert f(**{k: 63}) == echo.ESHAPE
    assert f(gate=FAKE, gate_tokens=2, ld_gate=63) == echo.ESHAPE
    assert f(gate=FAKE, gate_tokens=0) == echo.EINVAL
    assert f(post=2) == echo.EINVAL and f(post=0, w_post=FAKE) == echo.EINVAL
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert f(eps=eps) == echo.EINVAL
    assert f(res_scale=float("nan")) == echo.EINVAL and f(block_scale=float("inf")) == echo.EINVAL
    assert f(x=None) == echo.EINVAL and f(r_out=None, h=None) == echo.EINVAL
    assert f(h_dtype=echo.I8, h_scale=None) == echo.EINVAL
    assert f(h_dtype=echo.I8, h_scale=FAKE + 2) == echo.EALIGN
    for k in ("x", "r", "w_post", "w_pre", "r_out", "h"):
        assert f(**{k: FAKE + 1}) == echo.EALIGN
    assert f(gate=FAKE + 1, gate_tokens=4) == echo.EALIGN
    assert f(T=0, x=None) == 0 and f(H=0, x=None) == 0
    assert echo.lib().echo_block_norm(None, None) == echo.EINVAL


def test_block_norm_backward_refusals(host_only):
    def b(norm=None, **kw):
        g = echo.NormGrads()
        g.ld_dh = g.ld_dr_out = g.ld_dx = g.ld_dr = g.ld_dgate = 64
        g.dh_dtype = echo.BF16
        g.dh = g.dr_out = g.dx = g.dr = FAKE
        g.workspace, g.workspace_bytes = FAKE, echo.echo_block_norm_backward_workspace_bytes(4, 64)
        for k, v in kw.items():
            setattr(g, k, v)
        return rc_of(echo.echo_block_norm_backward, norm_args(**(norm or {})), g, stream=0)
    assert b(dh_dtype=echo.I8) == echo.EUNSUP and b(norm=dict(x_dtype=7)) == echo.EUNSUP
    for k in ("ld_dh", "ld_dr_out", "ld_dx", "ld_dr"):
        assert b(**{k: 63}) == echo.ESHAPE
    assert b(norm=dict(gate=FAKE, gate_tokens=1), dgate=FAKE, ld_dgate=3) == echo.ESHAPE
    assert b(dgate=FAKE) == echo.EINVAL                                  # no gate
    assert b(norm=dict(post=0), dw_post=FAKE) == echo.EINVAL             # no post norm
    assert b(norm=dict(r=None)) == echo.EINVAL                           # dr without r
    assert b(dh=None, dr_out=None) == echo.EINVAL
    for k in ("dh", "dr_out", "dx", "dr"):
        assert b(**{k: FAKE + 1}) == echo.EALIGN
    assert b(dw_pre=FAKE + 2) == echo.EALIGN and b(dw_post=FAKE + 2) == echo.EALIGN
    need = echo.echo_block_norm_backward_workspace_bytes(4, 64)
    assert need > 0
    assert b(workspace=None) == echo.EINVAL and b(workspace_bytes=need - 1) == echo.EINVAL
    assert b(workspace=FAKE + 4) == echo.EALIGN
    assert b(norm=dict(H=0)) == 0
    assert echo.echo_block_norm_backward_workspace_bytes(-1, 64) == 0
    assert echo.echo_block_norm_backward_workspace_bytes(4, (1 << 30) + 1) == 0
    assert echo.lib().echo_block_norm_backward(None, None, None) == echo.EINVAL


def test_binding_checks_tensors():
    """Shapes, types and strides that the C side cannot see are refused by the binding."""
    x = torch.zeros(6, 32, dtype=torch.bfloat16)
    w = torch.ones(32)
    ok = echo.make_norm_args(x, x, r_out=x, h=torch.zeros(6, 48, dtype=torch.int8), h_scale=torch.zeros(6), w_pre=w,
                             gate=torch.ones(2, 32), gate_tokens=4)
    assert (ok.T, ok.H, ok.ld_h, ok.gate_tokens, ok.h_dtype) == (6, 32, 48, 4, echo.I8)
    bad = [dict(r=torch.zeros(5, 32, dtype=torch.bfloat16)), dict(r=torch.zeros(32, 6).t()), dict(r=x.half()),
           dict(r=x, r_out=x.float()), dict(w_pre=torch.ones(31)), dict(w_pre=w, w_post=w.bfloat16()),
           dict(w_pre=torch.ones(64)[::2]), dict(gate=torch.ones(1, 32), gate_tokens=4),
           dict(gate=torch.ones(2, 32), gate_tokens=0), dict(h=torch.zeros(6, 31, dtype=torch.int8)),
           dict(h=torch.zeros(6, 32, dtype=torch.int8), h_scale=torch.zeros(5))]
    for kw in bad:
        with pytest.raises(ValueError):
            echo.make_norm_args(x, **kw)
    with pytest.raises(ValueError):
        echo.make_norm_grads(dh=x, dx=torch.zeros(5, 32))
    with pytest.raises(ValueError):
        echo.make_norm_grads(dh=x, dw_pre=torch.zeros(32, dtype=torch.bfloat16))
    a = echo.make_norm_args(x, x, gate=torch.ones(2, 32), gate_tokens=4)
    for kw in (dict(dr=x.float()), dict(dx=x.float()), dict(dgate=torch.zeros(3, 32))):
        with pytest.raises(ValueError):
            echo.echo_block_norm_backward(a, echo.make_norm_grads(dh=x, **kw), stream=0)


def test_plain_quantizer_edges():
    x = np.array([[0, 0, 0], [1e-40, -1e-41, 0], [127, -63.5, 0.5], [np.inf, 1, 2], [1, np.nan, 2], [3e38, -3e38, 1]], np.float32)
    q, s = ref.quantize_tokens(x)
    assert q[0].tolist() == [0, 0, 0] and s[0] == np.float32(2.0 ** -100) / np.float32(127)
    assert q[1].tolist() == [0, 0, 0]
    assert q[2].tolist() == [127, -64, 0] and s[2] == 1.0          # halves to even
    assert np.isnan(s[3]) and np.isnan(s[4]) and not q[3:5].any()
    assert q[5].tolist() == [127, -127, 0]


@pytest.mark.parametrize("post,gate_tokens,rho,beta", [(1, 2, 0.8, 0.5), (0, 0, 1.0, 1.0), (1, 1, 1.0, 0.3), (1, 100, 0.7, 1.0)])
def test_plain_gradients_against_differences(post, gate_tokens, rho, beta):
    """Central differences of L = sum(h dh) + sum(r' dr') in float64, step
    1e-6: truncation about step^2 and rounding about 2^-52 |L| / step, both
    below 1e-8 for values of order one."""
    rng = np.random.default_rng(7)
    T, H, eps, step = 5, 9, 1e-5, 1e-6
    v = dict(x=rng.standard_normal((T, H)), r=rng.standard_normal((T, H)), w_pre=1 + 0.2 * rng.standard_normal(H),
             w_post=1 + 0.2 * rng.standard_normal(H) if post else None,
             gate=rng.standard_normal((-(-T // gate_tokens), H)) if gate_tokens else None)
    dh, up = rng.standard_normal((T, H)), rng.standard_normal((T, H))

    def fwd(v):
        return ref.norm_forward(v["x"], v["r"], v["w_post"], v["w_pre"], v["gate"], gate_tokens, post, rho, beta, eps)

    def loss(v):
        f = fwd(v)
        return (f["h"] * dh).sum() + (f["rn"] * up).sum()

    got, _ = ref.norm_backward(fwd(v), v["x"], dh, up, v["gate"], gate_tokens, post, rho, beta)
    for name, t in v.items():
        if t is None:
            continue
        want = np.empty_like(t)
        for i in np.ndindex(*t.shape):
            sides = []
            for s in (step, -step):
                w = dict(v)
                w[name] = t.copy()
                w[name][i] += s
                sides.append(loss(w))
            want[i] = (sides[0] - sides[1]) / (2 * step)
        assert np.abs(got["d" + name] - want).max() < 1e-7, name
