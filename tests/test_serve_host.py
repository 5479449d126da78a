"""The serving operators without a GPU: the host's refusals, workspace sizes,
the binding's checks of tensors, and the plain quantizer against the oracle."""
import ctypes

import numpy as np
import pytest
import torch

import _serve_ref as ref
import oracle
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


@pytest.mark.parametrize("n", [1, 7, 32, 64, 128, 256])
def test_plain_quantizer_is_the_oracles(n):
    rng = np.random.default_rng(n)
    x = rng.standard_normal((64, n)).astype(np.float32) * np.exp2(rng.integers(-40, 40, (64, 1))).astype(np.float32)
    x[0], x[1], x[2], x[3] = 0, np.abs(x[1]), -np.abs(x[2]), 3e38 * np.sign(x[3])
    x[4:8] = np.clip(x[4:8], -6e4, 6e4).astype(np.float16)
    q, s, z = ref.quant4(x)
    for i in range(64):
        want = oracle.quantize_group(x[i], 4)
        np.testing.assert_array_equal(q[i], want[0], err_msg=str(i))
        assert (s[i], z[i]) == want[1:], i


def test_quantize_groups_refusals(host_only):
    def q(**kw):
        a = dict(x=FAKE, ldx=64, dt=echo.BF16, T=4, K=64, g=32, q=FAKE, ldq=32, p=FAKE, ldp=2) | kw
        return rc_of(echo.echo_quantize_groups, a["x"], a["ldx"], a["dt"], a["T"], a["K"], a["g"], a["q"], a["ldq"], a["p"], a["ldp"], stream=0)
    assert q(dt=echo.I8) == echo.EUNSUP and q(dt=echo.I4) == echo.EUNSUP
    assert q(g=16) == echo.EUNSUP and q(g=0) == echo.EUNSUP and q(g=96) == echo.EUNSUP and q(g=-32) == echo.EUNSUP
    assert q(T=-1) == echo.ESHAPE and q(K=-1) == echo.ESHAPE and q(K=(1 << 30) + 1) == echo.ESHAPE
    assert q(ldx=63) == echo.ESHAPE and q(ldq=31) == echo.ESHAPE and q(ldp=1) == echo.ESHAPE
    assert q(K=65, ldx=65, ldq=32, ldp=3) == echo.ESHAPE and q(K=65, ldx=65, ldq=33, ldp=2) == echo.ESHAPE
    assert q(x=None) == echo.EINVAL and q(q=None) == echo.EINVAL and q(p=None) == echo.EINVAL
    assert q(x=FAKE + 1) == echo.EALIGN and q(p=FAKE + 2) == echo.EALIGN and q(x=FAKE + 2, dt=echo.F32) == echo.EALIGN
    assert q(T=0, x=None) == 0 and q(K=0, x=None, q=None, p=None) == 0


def test_linear_int4_refusals(host_only):
    def f(**kw):
        a = dict(x=FAKE, ldx=64, xd=echo.BF16, w=FAKE, ldw=32, p=FAKE, ldp=2, g=32, bias=None, M=4, N=8, K=64, y=FAKE, ldy=8,
                 yd=echo.BF16, ws=FAKE, wb=1 << 40) | kw
        return rc_of(echo.echo_linear_int4, a["x"], a["ldx"], a["xd"], a["w"], a["ldw"], a["p"], a["ldp"], a["g"], a["bias"],
                     a["M"], a["N"], a["K"], a["y"], a["ldy"], a["yd"], a["ws"], a["wb"], stream=0)
    assert f(xd=echo.I8) == echo.EUNSUP and f(yd=echo.I4) == echo.EUNSUP and f(g=48) == echo.EUNSUP
    assert f(M=-1) == echo.ESHAPE and f(N=-1) == echo.ESHAPE and f(K=-1) == echo.ESHAPE
    assert f(ldx=63) == echo.ESHAPE and f(ldw=31) == echo.ESHAPE and f(ldp=1) == echo.ESHAPE and f(ldy=7) == echo.ESHAPE
    assert f(M=1 << 22, N=1 << 22, ldy=1 << 22) == echo.ESHAPE
    assert f(M=1 << 20, K=1 << 20, ldx=1 << 20, ldw=1 << 19, ldp=1 << 15) == echo.ESHAPE
    assert f(M=20, ws=None) == echo.EINVAL and f(M=20, wb=echo.echo_linear_int4_workspace_bytes(20, 8, 64, 32) - 1) == echo.EINVAL
    assert echo.echo_linear_int4_workspace_bytes(16, 8, 64, 32) == 0
    assert f(x=None) == echo.EINVAL and f(w=None) == echo.EINVAL and f(p=None) == echo.EINVAL and f(y=None) == echo.EINVAL
    assert f(x=FAKE + 1) == echo.EALIGN and f(p=FAKE + 2) == echo.EALIGN and f(bias=FAKE + 2) == echo.EALIGN
    assert f(y=FAKE + 1) == echo.EALIGN and f(ws=FAKE + 8) == echo.EALIGN
    assert f(M=0, x=None, y=None) == 0 and f(N=0, w=None, y=None) == 0
    for bad in ((-1, 8, 64, 32), (1, -8, 64, 32), (1, 8, -64, 32), (1, 8, 64, 33)):
        assert echo.echo_linear_int4_workspace_bytes(*bad) == 0


def a_cache(**kw):
    a = dict(pages=4, page_tokens=16, heads=2, width=64, ld_page=2048, ld_head=1024, ld_token=64, ld_scale_page=32,
             ld_scale_head=16, kind=echo.I8, k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE) | kw
    return echo.Cache(*(a[n] for n, _ in echo.Cache._fields_))


def a_seqs(**kw):
    a = dict(seqs=2, tokens=5, table_pages=3, ld_table=3, max_new=3, max_len=40, starts=FAKE, lens=FAKE, page_table=FAKE) | kw
    return echo.Seqs(*(a[n] for n, _ in echo.Seqs._fields_))


def write(c, s, k=FAKE, ld_k=128, v=FAKE, ld_v=128, dt=echo.BF16, fn="echo_cache_write"):
    return getattr(echo.lib(), fn)(ctypes.byref(c), ctypes.byref(s), k, ld_k, v, ld_v, dt, None)


def attend(c, s, ws=FAKE, wb=1 << 40, **kw):
    a = dict(cache=c, seqs=s, q_heads=4, ld_q=256, ld_out=256, window=0, causal=1, scale=0.125, q=FAKE, out=FAKE, lse=FAKE) | kw
    args = echo.AttentionArgs(*(a[n] for n, _ in echo.AttentionArgs._fields_))
    return echo.lib().echo_cache_attention(ctypes.byref(args), ws, wb, None)


CALLS = [write, lambda c, s: write(c, s, fn="echo_cache_read"), attend]


@pytest.mark.parametrize("call", CALLS, ids=["write", "read", "attention"])
def test_cache_and_sequence_refusals(host_only, call):
    c, s = a_cache, a_seqs
    assert call(c(kind=echo.F32), s()) == echo.EUNSUP and call(c(kind=7), s()) == echo.EUNSUP
    for bad in (dict(width=0), dict(width=60), dict(width=264, ld_token=264), dict(heads=0), dict(heads=70000), dict(page_tokens=0),
                dict(page_tokens=-1), dict(pages=-1), dict(pages=0), dict(pages=1 << 31), dict(ld_token=60), dict(ld_token=56),
                dict(ld_token=-64), dict(ld_head=1028), dict(ld_head=0), dict(ld_page=4), dict(ld_page=1 << 41), dict(ld_scale_page=-1),
                dict(ld_scale_head=1 << 41)):
        assert call(c(**bad), s()) == echo.ESHAPE, bad
    for bad in (dict(seqs=-1), dict(tokens=-1), dict(tokens=1 << 31), dict(seqs=1 << 31), dict(table_pages=-1), dict(ld_table=2),
                dict(max_new=-1), dict(max_len=-1)):
        assert call(c(), s(**bad)) == echo.ESHAPE, bad
    for bad in (dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None)):
        assert call(c(**bad), s()) == echo.EINVAL, bad
    for bad in (dict(starts=None), dict(lens=None), dict(page_table=None)):
        assert call(c(), s(**bad)) == echo.EINVAL, bad
    for bad in (dict(k=FAKE + 8), dict(v=FAKE + 4), dict(k_scale=FAKE + 2), dict(v_scale=FAKE + 1)):
        assert call(c(**bad), s()) == echo.EALIGN, bad
    for bad in (dict(starts=FAKE + 2), dict(lens=FAKE + 1), dict(page_table=FAKE + 2)):
        assert call(c(), s(**bad)) == echo.EALIGN, bad
    # no work: nothing is looked at
    none = dict(starts=None, lens=None, page_table=None)
    assert call(c(k=None, v=None, k_scale=None, v_scale=None), s(tokens=0, **none)) == 0
    assert call(c(pages=0, k=None), s(seqs=0, **none)) == 0


def test_cache_rows_refusals(host_only):
    for fn in ("echo_cache_write", "echo_cache_read"):
        w = lambda *a, **kw: write(*a, fn=fn, **kw)  # noqa: E731
        assert w(a_cache(), a_seqs(), dt=echo.I8) == echo.EUNSUP and w(a_cache(), a_seqs(), dt=-1) == echo.EUNSUP
        assert w(a_cache(), a_seqs(), ld_k=127) == echo.ESHAPE and w(a_cache(), a_seqs(), ld_v=127) == echo.ESHAPE
        assert w(a_cache(heads=40000), a_seqs(tokens=60000), ld_k=1 << 30, ld_v=1 << 30) == echo.ESHAPE
        assert w(a_cache(), a_seqs(), k=None) == echo.EINVAL and w(a_cache(), a_seqs(), v=None) == echo.EINVAL
        assert w(a_cache(), a_seqs(), k=FAKE + 1) == echo.EALIGN
        assert w(a_cache(), a_seqs(), v=FAKE + 2, dt=echo.F32) == echo.EALIGN
        assert getattr(echo.lib(), fn)(None, ctypes.byref(a_seqs()), FAKE, 128, FAKE, 128, 1, None) == echo.EINVAL


def test_attention_refusals(host_only):
    c, s = a_cache(), a_seqs()
    assert attend(c, s, q_heads=3) == echo.ESHAPE and attend(c, s, q_heads=0) == echo.ESHAPE and attend(c, s, q_heads=-2) == echo.ESHAPE
    assert attend(c, s, ld_q=255) == echo.ESHAPE and attend(c, s, ld_out=255) == echo.ESHAPE
    assert attend(c, a_seqs(tokens=1 << 30), ld_q=1 << 20, ld_out=1 << 20) == echo.ESHAPE          # rows past 31 bits
    assert attend(c, s, window=-1) == echo.EINVAL and attend(c, s, causal=2) == echo.EINVAL
    assert attend(c, s, scale=float("inf")) == echo.EINVAL and attend(c, s, scale=float("nan")) == echo.EINVAL
    assert attend(c, s, q=None) == echo.EINVAL and attend(c, s, out=None) == echo.EINVAL
    assert attend(c, s, q=FAKE + 1) == echo.EALIGN and attend(c, s, out=FAKE + 1) == echo.EALIGN
    assert attend(c, s, lse=FAKE + 2) == echo.EALIGN and attend(c, s, ws=FAKE + 8) == echo.EALIGN
    assert echo.lib().echo_cache_attention(None, FAKE, 0, None) == echo.EINVAL
    assert echo.lib().echo_cache_attention_workspace_bytes(None) == 0
    # a long sequence of one row is split, and its parts need room
    big = a_seqs(seqs=1, tokens=1, table_pages=4096, ld_table=4096, max_new=1, max_len=65536)
    args = echo.AttentionArgs(c, big, 4, 256, 256, 0, 1, 0.125, FAKE, FAKE, None)
    need = echo.echo_cache_attention_workspace_bytes(args)
    assert need > 0 and need % (4 * (64 * 4 + 8)) == 0
    assert attend(c, big, ws=None) == echo.EINVAL and attend(c, big, wb=need - 1) == echo.EINVAL


def test_binding_checks_tensors(host_only):
    mk = lambda *s, dt=torch.int8: torch.zeros(*s, dtype=dt)  # noqa: E731
    k, sc = mk(4, 2, 16, 64), mk(4, 2, 16, dt=torch.float32)
    c = echo.make_cache(k, k.clone(), sc, sc.clone())
    assert (c.pages, c.heads, c.page_tokens, c.width, c.kind) == (4, 2, 16, 64, echo.I8)
    assert (c.ld_page, c.ld_head, c.ld_token, c.ld_scale_page, c.ld_scale_head) == (2048, 1024, 64, 32, 16)
    k4, s4 = mk(4, 2, 16, 32, dt=torch.uint8), mk(4, 2, 16, 2, dt=torch.float16)
    c4 = echo.make_cache(k4, k4.clone(), s4, s4.clone())
    assert (c4.width, c4.kind, c4.ld_page, c4.ld_head, c4.ld_token, c4.ld_scale_page, c4.ld_scale_head) == (64, echo.I4, 2048, 1024, 64, 32, 16)
    tokens_first = mk(4, 16, 2, 64, dt=torch.bfloat16).permute(0, 2, 1, 3)
    cb = echo.make_cache(tokens_first, tokens_first)
    assert (cb.heads, cb.page_tokens, cb.ld_page, cb.ld_head, cb.ld_token) == (2, 16, 2048, 64, 128)
    for bad in (lambda: echo.make_cache(k, k[:3], sc, sc), lambda: echo.make_cache(k.half(), k.half()),
                lambda: echo.make_cache(k, k, sc, None), lambda: echo.make_cache(k, k, sc.half(), sc.half()),
                lambda: echo.make_cache(k, k, sc[:3], sc), lambda: echo.make_cache(tokens_first, tokens_first, sc, sc),
                lambda: echo.make_cache(k.transpose(2, 3), k.transpose(2, 3), sc, sc),
                lambda: echo.make_cache(k4, k4, sc, sc), lambda: echo.make_cache(k[0], k[0], sc, sc)):
        with pytest.raises(ValueError):
            bad()
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    s = echo.make_seqs(i(3), i(2), i(2, 5), 7, max_new=4, max_len=80)
    assert (s.seqs, s.tokens, s.table_pages, s.ld_table, s.max_new, s.max_len) == (2, 7, 5, 5, 4, 80)
    assert echo.make_seqs(i(3), i(2), i(2, 5), 7).max_new == 7
    for bad in (lambda: echo.make_seqs(i(2), i(2), i(2, 5), 7), lambda: echo.make_seqs(i(3).long(), i(2), i(2, 5), 7),
                lambda: echo.make_seqs(i(3), i(2), i(3, 5), 7), lambda: echo.make_seqs(i(3), i(2), i(5, 2).t(), 7)):
        with pytest.raises(ValueError):
            bad()
    q = mk(7, 256, dt=torch.bfloat16)
    a = echo.make_attention_args(c, s, q, q.clone(), 4, lse=mk(7, 4, dt=torch.float32))
    assert (a.q_heads, a.ld_q, a.ld_out, a.causal, a.window) == (4, 256, 256, 1, 0) and a.scale == 0.125
    for bad in (lambda: echo.make_attention_args(c, s, q[:6], q, 4), lambda: echo.make_attention_args(c, s, q.float(), q, 4),
                lambda: echo.make_attention_args(c, s, q, q, 8), lambda: echo.make_attention_args(c, s, q, q, 4, lse=mk(7, 3, dt=torch.float32)),
                lambda: echo.echo_cache_write(c, s, q[:, :128], q), lambda: echo.echo_cache_write(c, s, q[:, :128], q[:, :128].float()),
                lambda: echo.echo_cache_read(c, s, q[:6, :128], q[:6, :128])):
        with pytest.raises(ValueError):
            bad()
