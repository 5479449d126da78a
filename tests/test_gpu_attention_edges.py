"""Attention over the paged cache where its values end: slots that nothing was
written to, pages without a place, infinite scores, forms of odd pages and wide
heads.  Cases and checks are those of tests/test_gpu_attention.py."""
import pytest
import torch

from _helpers import DEV
from error_feedback_quant_amd import echo
from test_gpu_attention import Case
from test_gpu_cache import KINDS

pytestmark = pytest.mark.gpu


def same_bits(got, want):
    return all(torch.equal(g.view(torch.int16), w.view(torch.int16)) for g, w in zip(got, want))


def leave_page_0(c):
    """Page 0, which stands in for a page that is none, then holds no sequence's tokens."""
    at = c.table == 0
    if bool(at.any()):
        free = next(p for p in range(1, c.pages) if not bool((c.table == p).any()))
        for t in c.cache:
            if t is not None:
                t[free] = t[0]
        c.table[at] = free


def unseen_slots(c):
    """[pages, page tokens]: slots that no row of a sequence sees, as all of the rows together go over one run of tokens."""
    free = torch.ones(c.pages, c.page, dtype=torch.bool, device=DEV)
    for b in range(len(c.new)):
        for p in c.sees(b).any(0).nonzero()[:, 0].tolist():
            free[int(c.table[b, p // c.page]), p % c.page] = False
    return free


def mark(c, free, zero):
    """Every unseen slot without numbers: each byte of codes and scales 0xFF, or a 4-bit zero point of its own beside a scale of 1."""
    for t, s in zip(c.cache[:2], c.cache[2:]):
        raw = t.view(torch.uint8) if t.dtype != torch.bfloat16 else t.view(torch.int16)
        raw.permute(0, 2, 1, 3)[free] = 255 if raw.dtype == torch.uint8 else -1
        if s is None:
            continue
        if c.kind == "i4" and zero is not None:
            s.permute(0, 2, 1, 3)[free] = torch.tensor([1.0, zero], device=DEV).half()
        else:
            words = s.view(torch.int32)                        # a float, or a pair of binary16
            words.view(c.pages, c.heads, c.page).transpose(1, 2)[free] = -1


SLOTS = [  # D, page, new, len, window: of few rows and of many
    (128, 16, 4, 155, 0), (128, 16, 4, 155, 36), (128, 16, 93, 243, 0), (128, 16, 93, 243, 36), (128, 24, 93, 243, 36),
    (64, 16, 93, 241, 0), (64, 64, 93, 330, 100), (256, 16, 93, 250, 36), (80, 48, 93, 247, 5), (128, 16, 33, 33, 0)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", SLOTS, ids=lambda s: "-".join(map(str, s)))
def test_slots_that_no_row_sees(kind, shape):
    """Slots behind the last token, tokens before the first window (down to the tile's edge, which is staged with it), pages that are
    none where no row sees them, and page 0 in their place may hold anything: NaN, infinities, bytes that were never written."""
    D, page, new, L, window = shape
    c = Case(kind, 2, 2, D, page, [new], [L], window=window, order="tokens" if page == 16 else "heads")
    leave_page_0(c)
    clean = [x.clone() for x in c.check()]
    free = unseen_slots(c)
    assert bool(free.any(0).all()) and bool(free[0].all())
    unseen = [e for e in range(c.table.shape[1]) if int(c.table[0, e]) >= 0 and bool(free[int(c.table[0, e])].all())]
    for zero in (None, float("inf"), float("-inf"), float("nan")) if kind == "i4" else (None,):
        mark(c, free, zero)
        assert same_bits(c.run(), clean), zero
    for e in unseen:
        c.table[0, e] = -1
    assert same_bits(c.run(), clean)
    if window == 36 and L == 243 and page == 16:
        assert 6 in unseen                                     # tokens 96 .. 111: staged, the first that is seen is 115


@pytest.mark.parametrize("D", [64, 128])
def test_slots_that_no_row_sees_in_large_blocks(D):
    """The same where the blocks are of eight waves, beside a sequence of one row, over 4 bits."""
    new = [2500, 1, 1701]
    assert sum(new) * 64 >= 256 * 1024
    c = Case("i4", 2, 32, D, 64, new, [2513, 900, 2111], window=1000)
    leave_page_0(c)
    clean = [x.clone() for x in c.run()]
    assert bool(clean[0].isfinite().all())
    mark(c, unseen_slots(c), float("nan"))
    assert same_bits(c.run(), clean)


MINUS = [  # new, lens, window: the first rows of a prompt see few tokens; parts of long sequences
    ([1], [1], 0), ([3, 1], [3, 90], 1), ([90], [90], 0), ([90, 2], [400, 70], 1), ([100], [300], 17), ([2], [9000], 0), ([70], [5000], 0)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("shape", MINUS, ids=lambda s: "-".join(map(str, s[0] + s[1] + [s[2]])))
def test_infinite_queries(kind, sign, shape):
    """An infinity in q against keys of one sign: all scores are +infinity or all are -infinity, and exp(x - max) is NaN for both.  The
    other rows keep their bits."""
    new, lens, window = shape
    d = 5
    c = Case(kind, 1, 4, 128, 16, new, lens, window=window)
    if kind == "i4":
        k, s = c.cache[0], c.cache[2]                          # code 0 below a zero point of 8
        k[..., d // 2] &= 0xF0 if d % 2 == 0 else 0x0F
        s[..., 1] = 8.0
    else:
        c.cache[0][..., d] = -3
    clean, clean_lse = (x.clone() for x in c.check())
    hit = torch.zeros(c.T, 4, dtype=torch.bool, device=DEV)
    hit[::2, 1] = True
    c.q.view(c.T, 4, 128)[..., d][hit] = sign * float("inf")
    out, lse = c.run()
    assert bool(out[hit].isnan().all()) and bool(lse[hit].isnan().all())
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])


@pytest.mark.parametrize("new,L", [(1, 1), (1, 40), (2, 9000), (90, 90), (90, 500), (70, 5000)])
def test_scores_past_fp32(new, L):
    """Scores that overflow: NaN where one does upwards or all that a row sees do downwards; beside others one that overflows downwards
    has the weight 0, as any score far below the largest has."""
    c = Case("bf16", 1, 4, 128, 16, [new], [L])
    c.q.view(c.T, 4, 128)[..., 0] = 2.0 ** 100
    k = c.cache[0]
    for factor in (-1.0, 1.0):
        k[..., 0] = factor * 2.0 ** 40
        out, lse = c.run()
        assert bool(out.isnan().all()) and bool(lse.isnan().all())
    k[..., 0] = 0.0
    at = max(0, L - new)                                       # the first row's own token
    page, slot = int(c.table[0, at // 16]), at % 16
    k[page, :, slot, 0] = -(2.0 ** 10)                         # a score of about -2^107
    want = [x.clone() for x in c.run()]
    k[page, :, slot, 0] = -(2.0 ** 40)
    got = c.run()
    if at == 0:                                                # the first row sees nothing else
        assert bool(want[0].isfinite().all()) and bool(got[0][0].isnan().all()) and bool(got[1][0].isnan().all())
        got, want = [x[1:] for x in got], [x[1:] for x in want]
    assert same_bits(got, want) and bool(got[0].isfinite().all())


WIDE = [  # heads, G, D, page, new, lens, window, causal: heads wider than 128 over pages that end anywhere, few rows and many
    (1, 2, 256, 24, [1, 3], [100, 57], 0, True), (2, 4, 256, 7, [5], [3000], 0, True), (1, 16, 136, 40, [2], [500], 60, True),
    (2, 2, 256, 7, [50], [120], 33, True), (1, 1, 200, 5, [70], [71], 0, True), (1, 3, 256, 24, [100, 1, 40], [700, 300, 40], 0, True),
    (1, 4, 248, 1, [33], [90], 0, False), (2, 1, 256, 8, [300], [1111], 0, True)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", WIDE, ids=lambda s: "-".join(map(str, s[:4] + s[6:])))
def test_wide_heads_and_odd_pages(kind, shape):
    heads, G, D, page, new, lens, window, causal = shape
    Case(kind, heads, G, D, page, new, lens, window=window, causal=causal, order="tokens" if page == 7 else "heads").check()


@pytest.mark.parametrize("kind", ["bf16", "i8"])
@pytest.mark.parametrize("new,L", [(2, 300), (90, 300)])
@pytest.mark.parametrize("power", [100, -90])
def test_values_of_any_size(kind, new, L, power):
    """Values far from 1: weights of up to 2^8, and their sums, stay inside fp32."""
    c = Case(kind, 1, 4, 128, 16, [new], [L])
    (c.cache[1] if kind == "bf16" else c.cache[3]).mul_(2.0 ** power)
    c.check()
