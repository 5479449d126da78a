"""Writing the quantized paged cache and reading it back, bit for bit."""
import numpy as np
import pytest
import torch

import _serve_ref as ref
from _helpers import DEV, say
from error_feedback_quant_amd import echo

pytestmark = pytest.mark.gpu
KINDS = ["bf16", "i8", "i4"]


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def new_cache(kind, pages, heads, page, D, order="heads", fill=0x5B):
    """k, v and their scales, every byte marked; order "tokens" keeps a token's heads together."""
    dtype, width = {"bf16": (torch.bfloat16, D), "i8": (torch.int8, D), "i4": (torch.uint8, D // 2)}[kind]
    size = torch.empty(0, dtype=dtype).element_size()

    def marked(shape, dt, n):
        raw = torch.full((int(np.prod(shape)) * n,), fill, dtype=torch.uint8, device=DEV)
        return raw.view(dt).view(shape)

    def codes():
        if order == "tokens":
            return marked((pages, page, heads, width), dtype, size).permute(0, 2, 1, 3)
        return marked((pages, heads, page, width), dtype, size)

    def scales():
        if kind == "bf16":
            return None
        return marked((pages, heads, page) + ((2,) if kind == "i4" else ()), torch.float32 if kind == "i8" else torch.float16,
                      4 if kind == "i8" else 2)
    return codes(), codes(), scales(), scales()


def sequences(rng, new, lens, page, pages, wide=None):
    """starts, lens, a table of distinct pages, -1 behind each sequence's last page."""
    counts = [max(0, -(-n // page)) for n in lens]
    order = rng.permutation(pages)[:sum(counts)].tolist()
    wide = wide or max(counts + [1])
    table, at = np.full((len(lens), wide), -1, np.int32), 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    return i32(np.cumsum([0] + new).tolist()), i32(lens), i32(table.tolist())


def places(new, lens, table, page):
    """(row, page, slot) of every row that has a place."""
    t, got = 0, []
    for b, (n, l) in enumerate(zip(new, lens)):
        for i in range(n):
            pos = l - n + i
            if 0 <= pos < table.shape[1] * page and table[b, pos // page] >= 0:
                got.append((t + i, int(table[b, pos // page]), pos % page))
        t += n
    return got


def encode(kind, rows):
    """rows [n, D] fp32 -> codes and scales as they lie in the cache (numpy)."""
    if kind == "bf16":
        return torch.from_numpy(rows).bfloat16().view(torch.int16).numpy(), None
    if kind == "i8":
        q, s = ref.quant8(rows)
        return q, s.view(np.int32)
    q, s, z = ref.quant4(rows)
    return ref.pack4(q), np.stack([s, z], -1).view(np.int16)


def bits(t):
    """A tensor's elements as integers (numpy)."""
    to = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]
    return t.contiguous().view(to).cpu().numpy()


SHAPES = [  # heads, D, page, new, lens
    (8, 128, 64, [1], [1]), (2, 64, 16, [1, 1, 1], [17, 16, 15]), (1, 256, 128, [5, 0, 300], [5, 9, 777]), (3, 80, 1, [4, 2], [9, 2]),
    (4, 96, 24, [50, 1, 30], [100, 24, 30]), (1, 8, 5, [7, 3], [33, 3]), (5, 200, 32, [33], [65]), (8, 128, 16, [1] * 70, list(range(1, 71)))]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%d-%d-%d" % s[:3])
def test_write_and_read(kind, dtype, shape):
    heads, D, page, new, lens = shape
    order = "tokens" if heads % 2 else "heads"
    say("cache write/read", kind, dtype, shape[:3], order)
    rng = np.random.default_rng([heads, D, page])
    pages = sum(-(-n // page) for n in lens) + 2
    starts, dl, table = sequences(rng, new, lens, page, pages)
    cache = new_cache(kind, pages, heads, page, D, order)
    T, pad = sum(new), 3
    k, v = (torch.from_numpy(rng.standard_normal((T, heads * D + pad)).astype(np.float32) * 3).to(DEV).to(dtype)[:, :heads * D] for _ in range(2))
    k[0, :D] = 0
    before = [None if t is None else bits(t).copy() for t in cache]
    c, s = echo.make_cache(*cache), echo.make_seqs(starts, dl, table, T, max_new=max(new), max_len=max(lens))
    echo.echo_cache_write(c, s, k, v)
    torch.cuda.synchronize()
    where = places(new, lens, table.cpu().numpy(), page)
    assert len(where) == T
    want = before
    for i, x in enumerate((k, v)):
        rows = x.float().cpu().numpy().reshape(T, heads, D)
        codes, scales = encode(kind, rows.reshape(-1, D))
        codes = codes.reshape(T, heads, -1)
        for t, p, slot in where:
            want[i][p, :, slot] = codes[t]
            if scales is not None:
                want[2 + i][p, :, slot] = scales.reshape((T, heads) + scales.shape[1:])[t]
    for name, t, w in zip(("k", "v", "k_scale", "v_scale"), cache, want):
        if t is not None:
            np.testing.assert_array_equal(bits(t), w, err_msg=name)          # other slots keep their bytes
    # and back, in both types
    for out_dtype in (torch.float32, torch.bfloat16):
        outs = [torch.full((T + 1, heads * D + pad), 5.0, dtype=out_dtype, device=DEV) for _ in range(2)]
        echo.echo_cache_read(c, s, outs[0][:T, :heads * D], outs[1][:T, :heads * D])
        torch.cuda.synchronize()
        for i, o in enumerate(outs):
            assert bool((o[T] == 5).all()) and bool((o[:, heads * D:] == 5).all())
            idx = torch.tensor([(p, slot) for _, p, slot in where], device=DEV)
            held = cache[i][idx[:, 0], :, idx[:, 1]]
            sc = None if kind == "bf16" else cache[2 + i][idx[:, 0], :, idx[:, 1]]
            # (code - zero) * scale has at most 4 + 11 or 7 + 24 bits: in fp32 one rounding, of the exact product
            exact = ref.values(kind, held, sc, D).float().to(out_dtype)
            assert torch.equal(o[:T, :heads * D].reshape(T, heads, D), exact)


@pytest.mark.parametrize("kind", KINDS)
def test_tokens_without_a_place(kind):
    """Negative positions, entries past the table, page numbers that name no page: not written, read as NaN; rows of no
    sequence and sequences that leave the rows are not touched."""
    say("cache places", kind)
    heads, D, page, pages = 2, 64, 16, 4
    cache = new_cache(kind, pages, heads, page, D)
    before = [None if t is None else bits(t).copy() for t in cache]
    table = i32([[0, -1, 1], [pages, 2, 1 << 30], [3, 3, 3], [3, 3, 3]])
    # rows 0-2: positions -1, 0, 1; 3-6: 15 (page 4: none), 16, 17, 18; 7-9: 47, 48, 49; the last sequence leaves the rows
    starts, lens = i32([0, 3, 7, 10, 99]), i32([2, 19, 50, 40])
    T = 12
    x = torch.randn(T, heads * D, device=DEV)
    c, s = echo.make_cache(*cache), echo.make_seqs(starts, lens, table, T)
    echo.echo_cache_write(c, s, x, 2 * x)
    k, v = (torch.full((T, heads * D), 5.0, device=DEV) for _ in range(2))
    echo.echo_cache_read(c, s, k, v)
    torch.cuda.synchronize()
    placed = {1: (0, 0), 2: (0, 1), 4: (2, 0), 5: (2, 1), 6: (2, 2), 7: (3, 15)}
    for t in range(T):
        if t in placed:
            assert bool(k[t].isfinite().all()) and bool((v[t] - 2 * k[t]).abs().max() <= 0.02 * float(k[t].abs().max()) + 1e-6)
        elif t < 10:
            assert bool(k[t].isnan().all()) and bool(v[t].isnan().all()), t
        else:
            assert bool((k[t] == 5).all()) and bool((v[t] == 5).all()), t
    changed = {(p, sl) for p in range(pages) for sl in range(page) if not np.array_equal(bits(cache[0])[p, :, sl], before[0][p, :, sl])}
    assert changed == set(placed.values())


@pytest.mark.parametrize("kind", KINDS)
def test_rows_without_numbers(kind):
    """A row with an infinity or a NaN is NaN in the quantized caches and kept as it is in bfloat16; its neighbours are not touched."""
    say("cache no numbers", kind)
    cache = new_cache(kind, 2, 2, 16, 64)
    x = torch.randn(3, 128, device=DEV).bfloat16()
    x[1, 5], x[2, 127] = float("inf"), float("nan")
    c, s = echo.make_cache(*cache), echo.make_seqs(i32([0, 3]), i32([3]), i32([[1]]), 3)
    echo.echo_cache_write(c, s, x, x)
    k, v = (torch.empty(3, 128, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    echo.echo_cache_read(c, s, k, v)
    torch.cuda.synchronize()
    k = k.view(3, 2, 64)
    if kind == "bf16":
        assert torch.equal(k.view(torch.int16), x.view(3, 2, 64).view(torch.int16))
    else:
        assert bool(k[1, 0].isnan().all()) and bool(k[2, 1].isnan().all())
        assert bool(k[[0, 0, 1, 2], [0, 1, 1, 0]].isfinite().all())


def test_pages_past_32_bits():
    """Pages whose codes lie more than 2^32 elements behind the first."""
    say("cache far pages")
    heads, D, page = 1, 64, 16
    far = 6
    step = (1 << 32) // far + 4096
    raw = torch.zeros(far * step + 8192, dtype=torch.int8, device=DEV)
    k = raw.as_strided((far + 1, heads, page, D), (step // 8 * 8, page * D, D, 1))
    v = raw[page * D:].as_strided(k.shape, k.stride())
    sc = [torch.zeros(far + 1, heads, page, device=DEV) for _ in range(2)]
    c, s = echo.make_cache(k, v, *sc), echo.make_seqs(i32([0, 20]), i32([20]), i32([[far, far - 1]]), 20)
    x = torch.randn(20, D, device=DEV)
    echo.echo_cache_write(c, s, x, -x)
    q, ss = ref.quant8(x.cpu().numpy())
    torch.cuda.synchronize()
    np.testing.assert_array_equal(k[far, 0].cpu().numpy(), q[:16])
    np.testing.assert_array_equal(v[far - 1, 0, :4].cpu().numpy(), -q[16:])
    out = [torch.empty(20, D, device=DEV) for _ in range(2)]
    echo.echo_cache_read(c, s, *out)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(out[0].cpu().numpy(), q.astype(np.float32) * ss[:, None])
