"""Attention over the paged cache against 64 bits, within the bounds derived
in tests/_serve_ref.py."""
import numpy as np
import pytest
import torch

import _serve_ref as ref
from _helpers import DEV, say
from error_feedback_quant_amd import echo
from test_gpu_cache import KINDS, i32, new_cache, sequences

pytestmark = pytest.mark.gpu


class Case:
    """A filled cache, its sequences and queries, and the call over them."""

    def __init__(self, kind, heads, G, D, page, new, lens, seed=0, order="heads", window=0, causal=True, pad=0, spread=1.0, hints=None):
        say("attention", kind, "heads", heads, "x", G, "D", D, "page", page, "new", new[:6], "lens", lens[:6], order, window, causal, hints)
        rng = np.random.default_rng([seed, heads, G, D, page])
        gen = torch.Generator(device=DEV).manual_seed(seed + 1)
        self.kind, self.heads, self.G, self.D, self.page, self.new, self.lens = kind, heads, G, D, page, new, lens
        self.window, self.causal = window, causal
        self.pages = sum(max(0, -(-n // page)) for n in lens) + 2
        self.starts, self.dlens, self.table = sequences(rng, new, lens, page, self.pages)
        self.cache = new_cache(kind, self.pages, heads, page, D, order)
        n = self.pages * page
        x = [torch.randn(n, heads * D, generator=gen, device=DEV) * s for s in (1.0, 1.0)]
        x[0] *= 1 + 3 * (torch.rand(heads * D, generator=gen, device=DEV) < 0.05)
        every = echo.make_seqs(i32([0, n]), i32([n]), torch.arange(self.pages, dtype=torch.int32, device=DEV)[None], n)
        echo.echo_cache_write(echo.make_cache(*self.cache), every, *x)
        self.T = sum(new)
        self.q = (torch.randn(self.T, heads * G * D + pad, generator=gen, device=DEV) * 1.5 * spread).bfloat16()[:, :heads * G * D]
        self.pad, self.hints = pad, hints or {}
        self.scale = D ** -0.5

    def run(self, rows_more=2):
        T, H = self.T, self.heads * self.G
        self.out_buf = torch.full((T + rows_more, H * self.D + self.pad), 33.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((T, H), 44.0, device=DEV)
        seqs = echo.make_seqs(self.starts, self.dlens, self.table, T, **({"max_new": max(self.new), "max_len": max(self.lens)} | self.hints))
        args = echo.make_attention_args(echo.make_cache(*self.cache), seqs, self.q, self.out_buf[:T, :H * self.D], H, lse=self.lse,
                                        causal=self.causal, window=self.window, scale=self.scale)
        ws = torch.full((echo.echo_cache_attention_workspace_bytes(args),), 0xFF, dtype=torch.uint8, device=DEV)
        echo.echo_cache_attention(args, ws)
        torch.cuda.synchronize()
        assert bool((self.out_buf[T:] == 33).all()) and bool((self.out_buf[:, H * self.D:] == 33).all())
        return self.out_buf[:T, :H * self.D].view(T, H, self.D), self.lse

    def sequence(self, b):
        """k, v [heads, L, D] in float64 and the offsets that the bounds take."""
        L = max(0, self.lens[b])
        pages = self.table[b, :-(-L // self.page)].long()
        got = []
        for i in range(2):
            sc = self.cache[2 + i]
            v = ref.values(self.kind, self.cache[i][pages], None if sc is None else sc[pages], self.D)
            got.append(v.transpose(0, 1).reshape(self.heads, -1, self.D)[:, :L])
        offs = [None] * self.heads
        if self.kind == "i4":
            o = [((16 + t[pages][..., 1].double()) * t[pages][..., 0].double()).transpose(0, 1).reshape(self.heads, -1)[:, :L] for t in self.cache[2:]]
            offs = [(o[0][h], o[1][h]) for h in range(self.heads)]
        return got[0], got[1], offs

    def sees(self, b):
        n, L = self.new[b], max(0, self.lens[b])
        pos = torch.arange(self.lens[b] - n, self.lens[b], device=DEV)[:, None]
        j = torch.arange(L, device=DEV)[None]
        s = (j <= pos) if self.causal else (j < L).expand(n, L)
        return s & (j > pos - self.window) if self.window else s

    def check(self, only=None):
        out, lse = self.run()
        t = 0
        for b, n in enumerate(self.new):
            if n and (only is None or b in only):
                k, v, offs = self.sequence(b)
                sees = self.sees(b)
                for h in range(self.heads):
                    for g in range(self.G):
                        hq = h * self.G + g
                        q = self.q[t:t + n].view(n, -1, self.D)[:, hq].double()
                        w, wl, tol, tl = (x.to(DEV) for x in ref.attention(q, k[h], v[h], sees, self.scale, offs[h]))
                        bad = ref.outside(out[t:t + n, hq], w, tol)
                        assert not bool(bad.any()), (b, hq, int(bad.sum()), bad.nonzero()[:4].tolist(),
                                                     out[t:t + n, hq][bad][:4].tolist(), w[bad][:4].tolist())
                        gl, empty = lse[t:t + n, hq].double(), ~sees.any(1)
                        assert torch.equal(gl == -torch.inf, empty)
                        off = ((gl - wl).abs() > tl) & ~empty
                        assert not bool(off.any()), (b, hq, gl[off][:4].tolist(), wl[off][:4].tolist())
            t += n
        return out, lse


ONES = [  # heads, G, D, page, lens of single tokens
    (2, 4, 128, 64, [1]), (2, 4, 128, 16, [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 500]), (1, 1, 64, 16, [700, 3]),
    (8, 8, 64, 32, [100]), (1, 16, 128, 128, [1000]), (2, 3, 256, 16, [257, 40]), (1, 5, 80, 24, [190, 24]), (3, 2, 96, 1, [77]),
    (1, 32, 128, 16, [300]), (2, 2, 8, 5, [64, 1]), (1, 7, 200, 48, [400]), (1, 2, 120, 7, [150])]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", ONES, ids=lambda s: "-".join(map(str, s[:4])))
def test_single_tokens(kind, shape):
    heads, G, D, page, lens = shape
    Case(kind, heads, G, D, page, [1] * len(lens), lens, order="tokens" if G % 2 else "heads", pad=G % 4).check()


CHUNKS = [  # heads, G, D, page, new, lens, window, causal
    (2, 4, 128, 64, [5, 1, 0, 9], [5, 70, 8, 200], 0, True), (1, 8, 64, 16, [16, 3], [40, 3], 0, True),
    (2, 2, 128, 16, [130], [130], 0, True), (1, 4, 128, 32, [200, 1, 77], [333, 900, 77], 0, True),
    (2, 1, 256, 16, [40, 2], [100, 2], 0, True), (1, 2, 80, 24, [60], [91], 0, True), (1, 3, 96, 1, [33], [70], 0, True),
    (2, 4, 128, 64, [50, 4], [300, 64], 64, True), (1, 8, 64, 16, [7, 100], [500, 129], 1, True), (2, 2, 128, 16, [70], [400], 33, True),
    (2, 2, 128, 16, [20, 3], [150, 3], 0, False), (1, 4, 64, 16, [9], [200], 50, False), (1, 1, 128, 5, [300], [301], 100, True),
    (1, 2, 8, 3, [65], [65], 0, True), (4, 1, 128, 128, [257], [1000], 0, True), (1, 4, 120, 16, [129, 127], [129, 300], 0, True)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", CHUNKS, ids=lambda s: "-".join(map(str, s[:4] + s[6:])))
def test_chunks(kind, shape):
    heads, G, D, page, new, lens, window, causal = shape
    Case(kind, heads, G, D, page, new, lens, window=window, causal=causal, order="tokens" if page == 16 else "heads", pad=len(new) % 2).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new", [1, 40])
def test_rows_that_see_nothing(kind, new):
    """Positions before the first token (lens below the new tokens, none at all): 0 and -infinity."""
    c = Case(kind, 2, 4, 128, 16, [new, new + 1, new, 3], [0, new - 1, new + 3, -5])
    out, lse = c.check()
    assert bool((out[:new] == 0).all()) and bool((lse[:new] == -torch.inf).all())
    assert bool((out[-3:] == 0).all()) and bool((lse[-3:] == -torch.inf).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_sequences_in_parts(kind, D):
    """Tens of thousands of tokens, whose parts are joined; the same bits every time."""
    c = Case(kind, 1, 2, D, 64, [1, 1, 3], [40000, 900, 20001])
    out, lse = c.check()
    again = c.run()
    assert torch.equal(again[0].view(torch.int16), out.view(torch.int16)) and torch.equal(again[1].view(torch.int32), lse.view(torch.int32))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new", [[1, 1, 1], [30, 1, 64]])
def test_hints_only_split_the_work(kind, new):
    """max_new and max_len may be anything: the rows are computed all the same."""
    lens = [100, 3000, 700]
    for hints in (dict(max_new=0, max_len=0), dict(max_new=1, max_len=1), dict(max_new=2, max_len=1 << 40), dict(max_new=1 << 40, max_len=64),
                  dict(max_new=None, max_len=None)):
        Case(kind, 2, 4, 128, 16, new, lens, hints=hints).check()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new", [4, 90])
@pytest.mark.parametrize("window", [0, 40])
def test_values_behind_the_mask(kind, new, window):
    """Tokens without numbers that a row does not see, in any element: later tokens of the chunk, slots behind the last token, tokens
    before the window.  Rows that see one are NaN there; the others keep their bits."""
    L, D = 150 + new, 128
    c = Case(kind, 2, 2, D, 16, [new], [L], window=window)
    clean, clean_lse = (x.clone() for x in c.check())
    k, v, ks, vs = c.cache
    late = L - new // 2                                   # a position inside the chunk
    page, slot = int(c.table[0, late // 16]), late % 16
    behind = int(c.table[0, (L - 1) // 16])
    for b in (float("nan"), float("inf")):
        for t, s in ((k, ks), (v, vs)):
            if kind == "bf16":
                t[page, :, slot, 77] = b
                t[behind, :, (L - 1) % 16 + 1:] = b
                if window:
                    t[int(c.table[0, 0]), :, :] = -b
            else:
                s[page, :, slot] = float("nan") if kind == "i8" else torch.tensor([float("nan"), 0.0], device=DEV).half()
                if (L - 1) % 16 + 1 < 16:
                    s[behind, :, (L - 1) % 16 + 1:] = float("nan")
                if window:
                    s[int(c.table[0, 0])] = float("nan")
        out, lse = c.run()
        pos = torch.arange(L - new, L, device=DEV)
        sees = (pos >= late) & (pos < late + window if window else pos >= 0)
        assert torch.equal(out[~sees].view(torch.int16), clean[~sees].view(torch.int16))
        assert torch.equal(lse[~sees], clean_lse[~sees])
        assert bool(out[sees].isnan().any(-1).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("new", [1, 3, 100])
def test_pages_that_are_none(kind, new):
    """Page numbers that name no page, and tokens past the table: rows that see such a token are NaN, the others keep their bits."""
    c = Case(kind, 2, 4, 128, 16, [new, new], [200 + new, 210])
    clean, clean_lse = (x.clone() for x in c.check())
    c.window = 30                                          # rows that do not see the page
    windowed = [x.clone() for x in c.check()]
    for none in (c.pages, -1, -(1 << 31)):
        c.table[0, 3], c.window = none, 0
        out, lse = c.run()
        assert bool(out[:new].isnan().all()) and torch.equal(out[new:], clean[new:]) and torch.equal(lse[new:], clean_lse[new:])
        c.window = 30
        assert all(torch.equal(x, y) for x, y in zip(c.run(), windowed))
    c.window = 0
    c.table = c.table[:, :13].contiguous()                 # 208 tokens
    out, lse = c.run()
    assert bool(out[:new].isnan().all())
    pos = torch.arange(210 - new, 210, device=DEV)
    assert bool(out[new:][pos >= 208].isnan().all())
    # a smaller table may split otherwise: each of the two is off by a step of the weights (below max |v| < 8) and one of the output
    got, want = out[new:][pos < 208].float(), clean[new:][pos < 208].float()
    assert bool(((got - want).abs() <= 2.1 * ref.BF * (8 + want.abs())).all())


def test_queries_without_numbers_and_large_scores():
    c = Case("i8", 2, 4, 128, 16, [40], [90])
    clean, _ = (x.clone() for x in c.check())
    c.q[7, 128 * 3 + 5] = float("inf")
    c.q[9, 0] = float("nan")
    out, lse = c.run()
    hit = torch.zeros(40, 8, dtype=torch.bool, device=DEV)
    hit[7, 3], hit[9, 0] = True, True
    assert bool(out[hit].isnan().all()) and torch.equal(out[~hit], clean[~hit])
    # scores of a few thousand: one token takes everything, without overflow
    Case("bf16", 1, 4, 128, 16, [30, 1], [300, 2000], spread=300.0).check()
    Case("i8", 1, 4, 128, 16, [30, 1], [300, 2000], spread=300.0).check()


def test_sequences_that_leave_the_rows():
    """Starts that the rows do not hold: those sequences are not taken, and nothing outside is touched."""
    c = Case("i8", 2, 4, 128, 16, [3, 5, 2], [60, 70, 80])
    clean, _ = (x.clone() for x in c.check())
    good = c.starts.clone()
    for bad in ([0, 3, 99, 10], [0, 3, 8, 1 << 30], [-7, 3, 8, 10], [0, 3, 2, 10], [-(1 << 31), (1 << 31) - 1, 0, 5]):
        c.starts = i32([max(min(v, (1 << 31) - 1), -(1 << 31)) for v in bad])
        out, _ = c.run()
        if bad[:2] == [0, 3]:
            n = min(3, bad[2])                             # rows of the first sequence alone
            assert torch.equal(out[:n], clean[:n])
    c.starts = good
    assert torch.equal(c.run()[0], clean)


def test_far_pages():
    """Pages more than 2^32 elements behind the first."""
    heads, D, page, far = 1, 64, 16, 6
    say("attention far pages")
    step = ((1 << 32) // far + 4096) // 8 * 8
    raw = torch.randint(-127, 128, (2 * page * D,), dtype=torch.int8, device=DEV)
    big = torch.zeros(far * step + 8192, dtype=torch.int8, device=DEV)
    k = big.as_strided((far + 1, heads, page, D), (step, page * D, D, 1))
    v = big[page * D:].as_strided(k.shape, k.stride())
    k[far, 0], v[far, 0] = raw[:page * D].view(page, D), raw[page * D:].view(page, D)
    sc = [torch.full((far + 1, heads, page), 0.01, device=DEV) for _ in range(2)]
    for n in (1, 12):
        q = torch.randn(n, 4 * D, device=DEV).bfloat16()
        near = [t[far:].contiguous() for t in (k, v)] + [t[far:].contiguous() for t in sc]
        outs = []
        for cache, table in (((k, v, *sc), far), (near, 0)):
            seqs = echo.make_seqs(i32([0, n]), i32([15]), i32([[table]]), n, max_new=n, max_len=15)
            out = torch.empty_like(q)
            args = echo.make_attention_args(echo.make_cache(*cache), seqs, q, out, 4)
            echo.echo_cache_attention(args, torch.empty(echo.echo_cache_attention_workspace_bytes(args), dtype=torch.uint8, device=DEV))
            outs.append(out)
        torch.cuda.synchronize()
        assert torch.equal(*outs) and bool(outs[0].isfinite().all())


@pytest.mark.parametrize("kind", KINDS)
def test_a_serving_step_in_a_graph(kind):
    """Write and attention over several parts captured together on a side stream and replayed beside eager work, each replay with other
    lengths, pages and inputs, against the eager calls."""
    say("attention in a graph", kind)
    heads, G, D, page, B = 2, 4, 128, 16, 3
    pages, wide = 700, 220
    cache = new_cache(kind, pages, heads, page, D, fill=0)
    rng = np.random.default_rng(5)
    gen = torch.Generator(device=DEV).manual_seed(1)
    n = pages * page
    every = echo.make_seqs(i32([0, n]), i32([n]), torch.arange(pages, dtype=torch.int32, device=DEV)[None], n)
    c = echo.make_cache(*cache)
    echo.echo_cache_write(c, every, *(torch.randn(n, heads * D, generator=gen, device=DEV) for _ in range(2)))
    T = 4
    starts, lens, table = i32([0, 1, 2, 4]), i32([1, 1, 2]), torch.zeros(B, wide, dtype=torch.int32, device=DEV)
    k, v = (torch.empty(T, heads * D, device=DEV).bfloat16() for _ in range(2))
    q = torch.empty(T, heads * G * D, device=DEV).bfloat16()
    out, lse = torch.empty_like(q), torch.empty(T, heads * G, device=DEV)
    seqs = echo.make_seqs(starts, lens, table, T, max_new=2, max_len=wide * page)
    args = echo.make_attention_args(c, seqs, q, out, heads * G, lse=lse)
    ws = torch.empty(echo.echo_cache_attention_workspace_bytes(args), dtype=torch.uint8, device=DEV)
    assert ws.numel() > 0

    def step():
        echo.echo_cache_write(c, seqs, k, v)
        echo.echo_cache_attention(args, ws)

    def inputs(i):
        order = rng.permutation(pages)
        table.copy_(torch.from_numpy(order[:B * wide].reshape(B, wide).astype(np.int32)))
        lens.copy_(i32([1 + 7 * i, 3000 + i, 2 + 400 * i]))
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, generator=gen, device=DEV))

    inputs(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(4):
        inputs(i)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        out.zero_()
        step()                                             # the same write again, then the eager attention
        torch.cuda.synchronize()
        assert torch.equal(out, got[0]) and torch.equal(lse, got[1]), i
        assert bool(out.float().abs().sum() > 0)


def test_two_streams_at_once():
    """Two calls that overlap in time, each with a workspace of its own."""
    a, b = Case("i8", 2, 4, 128, 16, [1, 1], [9000, 300], seed=1), Case("i4", 2, 4, 128, 16, [1, 2], [7000, 20], seed=2)
    want = [tuple(x.clone() for x in c.run()) for c in (a, b)]
    calls, lses = [], []
    for c in (a, b):
        seqs = echo.make_seqs(c.starts, c.dlens, c.table, c.T, max_new=max(c.new), max_len=max(c.lens))
        out, lse = torch.zeros(c.T, 8 * 128, dtype=torch.bfloat16, device=DEV), torch.zeros(c.T, 8, device=DEV)
        args = echo.make_attention_args(echo.make_cache(*c.cache), seqs, c.q, out, 8, lse=lse)
        ws = torch.empty(echo.echo_cache_attention_workspace_bytes(args), dtype=torch.uint8, device=DEV)
        lses.append(lse)
        calls.append((args, ws, out, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for args, ws, _, st in calls:
            echo.echo_cache_attention(args, ws, stream=st)
    torch.cuda.synchronize()
    for (w, wl), (_, _, out, _), lse in zip(want, calls, lses):
        assert torch.equal(out.view(w.shape), w) and torch.equal(lse, wl)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,window,causal", [(64, 0, True), (128, 0, True), (128, 700, True), (64, 300, False), (96, 0, True)])
def test_many_rows(kind, D, window, causal):
    """Enough rows for the blocks of eight waves, beside a sequence of one row."""
    new = [2500, 1, 1700]
    assert sum(new) * 64 >= 256 * 1024
    Case(kind, 2, 32, D, 64, new, [2500, 900, 2111], window=window, causal=causal).check()
