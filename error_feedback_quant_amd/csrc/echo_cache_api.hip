// echo_cache_api.hip — host side of the quantized paged cache and of attention
// over it: argument checks and launches; semantics, layouts and error
// behaviour are specified in include/echo.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "echo.h"
#include "echo_attention.hpp"
#include "echo_host.hpp"

namespace {

using echo::aligned16;
using echo::aligned_elem;
using echo::aligned_to;
using echo::bad_dim;
using echo::bad_ld;
using echo::check_launch;
using echo::float_dtype;
using echo::grid_of;
using echo::kMaxRows;

constexpr int64_t kMaxCacheRows = int64_t(1) << 26;       // of a call: 32 lanes each, keys and values, in 32 bits of threads
constexpr int64_t kMaxStride = int64_t(1) << 40;        // of pages and heads, in elements
constexpr int64_t kMaxLen = (int64_t(1) << 31) - (1 << 12);     // positions and the tiles behind them stay in 31 bits
constexpr int64_t kCus = 256;

int check_cache(const echo_cache& c)
{
    if (c.kind != ECHO_BF16 && c.kind != ECHO_I8 && c.kind != ECHO_I4) return ECHO_EUNSUP;
    if (bad_dim(c.pages, kMaxRows) || bad_dim(c.page_tokens, kMaxRows) || bad_dim(c.heads, 65535)) return ECHO_ESHAPE;
    if (c.page_tokens < 1 || c.heads < 1 || c.width < 8 || c.width > 256 || c.width % 8) return ECHO_ESHAPE;
    if (bad_dim(c.ld_page, kMaxStride) || bad_dim(c.ld_head, kMaxStride) || bad_dim(c.ld_token, kMaxStride) ||
        c.ld_page % 8 || c.ld_head % 8 || c.ld_token % 8)
        return ECHO_ESHAPE;
    // a stride that is used at all steps over a row
    if ((c.page_tokens > 1 && c.ld_token < c.width) || (c.heads > 1 && c.ld_head < c.width) ||
        (c.pages > 1 && c.ld_page < c.width))
        return ECHO_ESHAPE;
    if (c.kind != ECHO_BF16 && (bad_dim(c.ld_scale_page, kMaxStride) || bad_dim(c.ld_scale_head, kMaxStride)))
        return ECHO_ESHAPE;
    return ECHO_OK;
}

int check_seqs(const echo_seqs& s)
{
    if (bad_dim(s.seqs, kMaxRows) || bad_dim(s.tokens, kMaxRows) || bad_dim(s.table_pages, kMaxRows)) return ECHO_ESHAPE;
    if (s.max_new < 0 || s.max_len < 0 || bad_ld(s.ld_table, s.seqs, s.table_pages)) return ECHO_ESHAPE;
    return ECHO_OK;
}

bool no_work(const echo_seqs& s) { return s.seqs == 0 || s.tokens == 0; }

// pointers of a call that has work
int check_pointers(const echo_cache& c, const echo_seqs& s)
{
    if (!c.k || !c.v || !s.starts || !s.lens || (s.table_pages && !s.page_table)) return ECHO_EINVAL;
    if (c.pages < 1) return ECHO_ESHAPE;
    if (c.kind != ECHO_BF16 && (!c.k_scale || !c.v_scale)) return ECHO_EINVAL;
    if (!aligned16(c.k) || !aligned16(c.v) || !aligned_to(s.starts, 4) || !aligned_to(s.lens, 4) ||
        !aligned_to(s.page_table, 4))
        return ECHO_EALIGN;
    if (c.kind != ECHO_BF16 && (!aligned_to(c.k_scale, 4) || !aligned_to(c.v_scale, 4))) return ECHO_EALIGN;
    return ECHO_OK;
}

echo::CacheView cache_view(const echo_cache& c)
{
    echo::CacheView v;
    std::memset(&v, 0, sizeof(v));
    v.k = (uint8_t*)c.k; v.v = (uint8_t*)c.v; v.ks = (uint32_t*)c.k_scale; v.vs = (uint32_t*)c.v_scale;
    v.ld_page = c.ld_page; v.ld_head = c.ld_head; v.ld_token = c.ld_token;
    v.ld_sp = c.ld_scale_page; v.ld_sh = c.ld_scale_head;
    v.pages = (uint32_t)c.pages; v.page_tokens = (uint32_t)c.page_tokens;
    v.heads = (int)c.heads; v.width = (int)c.width;
    return v;
}

echo::SeqView seq_view(const echo_seqs& s, const echo_cache& c)
{
    echo::SeqView v;
    std::memset(&v, 0, sizeof(v));
    v.starts = s.starts; v.lens = s.lens; v.table = s.page_table;
    v.ld_table = s.ld_table; v.table_pages = s.table_pages;
    v.capacity = std::min(s.table_pages * c.page_tokens, kMaxLen);          // the product is below 2^62
    v.seqs = (int)s.seqs; v.tokens = s.tokens;
    return v;
}

template <int KIND, int L, int U, bool WRITE>
void cache_io_go(const echo::CacheIoArgs& a, bool bf16, hipStream_t st)
{
    const int64_t rows = echo::kBlock / L * U;              // of a block
    const dim3 grid((unsigned)((a.rows + rows - 1) / rows), 2), block(echo::kBlock);
    if constexpr (WRITE) {
        if (bf16) hipLaunchKernelGGL((echo::cache_write_kernel<KIND, L, U, true>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((echo::cache_write_kernel<KIND, L, U, false>), grid, block, 0, st, a);
    } else {
        if (bf16) hipLaunchKernelGGL((echo::cache_read_kernel<KIND, L, U, true>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((echo::cache_read_kernel<KIND, L, U, false>), grid, block, 0, st, a);
    }
}

template <int KIND, bool WRITE>
void cache_io_sized(const echo::CacheIoArgs& a, bool bf16, hipStream_t st)
{
    const int L = a.c.width <= 64 ? 8 : (a.c.width <= 128 ? 16 : 32);
    // Four rows on their way where there are threads for all CUs several times
    // over, else one (us for a write and a read of 8 heads of 128 in 8 bits, one
    // row and four: 512 tokens 7.2, 8.5, 1024 9.0, 9.1, 2048 12.9, 10.9, 8192
    // 36.6, 23.7).
    const bool many = a.rows * L >= 4 * 256 * kCus;
    auto go = [&](auto l) {
        if (many) cache_io_go<KIND, decltype(l)::value, 4, WRITE>(a, bf16, st);
        else cache_io_go<KIND, decltype(l)::value, 1, WRITE>(a, bf16, st);
    };
    if (L == 8) go(std::integral_constant<int, 8>{});
    else if (L == 16) go(std::integral_constant<int, 16>{});
    else go(std::integral_constant<int, 32>{});
}

template <bool WRITE>
int cache_io(const echo_cache* c, const echo_seqs* s, void* k, int64_t ld_k, void* v, int64_t ld_v, int dtype, void* stream)
{
    if (!c || !s) return ECHO_EINVAL;
    if (!float_dtype(dtype)) return ECHO_EUNSUP;
    int rc = check_cache(*c);
    if (rc) return rc;
    if ((rc = check_seqs(*s))) return rc;
    if (s->tokens * c->heads > kMaxCacheRows || bad_ld(ld_k, s->tokens, c->heads * c->width) ||
        bad_ld(ld_v, s->tokens, c->heads * c->width))
        return ECHO_ESHAPE;
    if (no_work(*s)) return ECHO_OK;
    if ((rc = check_pointers(*c, *s))) return rc;
    if (!k || !v) return ECHO_EINVAL;
    if (!aligned_elem(k, dtype) || !aligned_elem(v, dtype)) return ECHO_EALIGN;
    echo::CacheIoArgs a;
    std::memset(&a, 0, sizeof(a));
    a.c = cache_view(*c);
    a.s = seq_view(*s, *c);
    a.x[0] = k; a.x[1] = v; a.ld[0] = ld_k; a.ld[1] = ld_v;
    a.rows = s->tokens * c->heads;
    const bool bf16 = dtype == ECHO_BF16;
    const hipStream_t st = (hipStream_t)stream;
    switch (c->kind) {
    case ECHO_BF16: cache_io_sized<echo::kCacheBf16, WRITE>(a, bf16, st); break;
    case ECHO_I8: cache_io_sized<echo::kCacheI8, WRITE>(a, bf16, st); break;
    default: cache_io_sized<echo::kCacheI4, WRITE>(a, bf16, st); break;
    }
    return check_launch();
}

// -------------------------------------------------------------- attention --

// How a call is split.
struct AttnPlan {
    bool few, tile;         // which kernels run; with both, a sequence of few rows is the former's
    int64_t few_tiles;      // row tiles of a sequence with a block of their own
    int tile_waves;         // of a block of the other kernel, 32 rows each
    int64_t tile_tiles;     // row tiles of all sequences together, at most
    int few_splits, tile_splits;        // parts of a row's tokens
    size_t few_ml, tile_o, tile_ml, total;      // of the workspace: the parts' sums of v, and their m and l
};

// Up to kFewAlone rows of a sequence and head go to the kernel for few rows (24
// sequences of up to 5 tokens and 8 heads: 14.0 us, with the other kernel from 16
// rows on 25.1).  Beside longer sequences, those of up to kFewBeside rows do (512
// tokens beside 7 single ones: 147 us, all in the other kernel 180).
constexpr int64_t kFewAlone = 64, kFewBeside = 16;
// Tokens are split until there are so many blocks, in parts of that length at
// least.  Few rows: 64 tokens over up to 16384 219 us with half as many blocks,
// 185 so, 186 with twice as many.  The other kernel, in the call above: 209, 147
// and 160; parts of half the length make no difference.
constexpr int64_t kFewBlocks = 8 * kCus, kFewBesideBlocks = 4 * kCus, kFewPart = 256, kTileBlocks = 2 * kCus, kTilePart = 512, kMostSplits = 64;
constexpr int64_t kMostBlocks = int64_t(1) << 22;       // their threads are 32 bits

constexpr int64_t kMaxQueries = int64_t(1) << 29;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Parts of `len` tokens so that `blocks` become `want`, none shorter than `part`.
int64_t splits_for(int64_t blocks, int64_t want, int64_t len, int64_t part)
{
    const int64_t s = std::min({ceil_div(want, std::max<int64_t>(1, blocks)), ceil_div(len, part), kMostSplits});
    return std::max<int64_t>(1, std::min(s, kMostBlocks / std::max<int64_t>(1, blocks)));
}

// 16 tokens of a page together, at 32-bit offsets from the first
bool paged16(const echo_cache& c) { return c.page_tokens % 16 == 0 && c.ld_token < int64_t(1) << 26; }

AttnPlan attn_plan(const echo_attention_args& p)
{
    AttnPlan n = {};
    const int64_t G = p.q_heads / p.cache.heads, T = p.seqs.tokens, H = p.cache.heads, pairs = p.seqs.seqs * H;
    const int64_t most_new = std::max<int64_t>(1, std::min(p.seqs.max_new, T));
    n.tile = most_new * G > kFewAlone;
    n.few = !n.tile || p.seqs.seqs > 1;
    // tokens that a row tile sees at most
    int64_t len = std::min(p.seqs.max_len, p.seqs.table_pages * p.cache.page_tokens);
    const int64_t seen = p.window > 0 ? std::min(p.window, len) : len;
    auto part = [&](int64_t rows, int64_t splits, size_t& o, size_t& ml) {
        if (splits <= 1) return;
        o = (n.total + 255) & ~(size_t)255;
        ml = o + (size_t)(rows * splits * p.cache.width * 4);
        n.total = ml + (size_t)(rows * splits * 8);
    };
    if (n.few) {
        n.few_tiles = std::max<int64_t>(1, std::min(ceil_div(n.tile ? kFewBeside : most_new * G, echo::kFewRows), kMostBlocks / pairs));
        const int64_t blocks = n.few_tiles * pairs;
        n.few_splits = (int)splits_for(blocks, n.tile ? kFewBesideBlocks : kFewBlocks, std::min(len, seen + echo::kFewRows / G + 1), kFewPart);
        size_t first = 0;
        part(n.tile ? pairs * kFewBeside : T * p.q_heads, n.few_splits, first, n.few_ml);
    }
    if (n.tile) {
        // Eight waves share what they stage, where there are blocks for all CUs
        // several times over (8192 tokens over 8192, 8 bits: 698 us with four
        // waves, 631 with eight; 512 tokens beside 7 sequences: 147 and 158).
        n.tile_waves = paged16(p.cache) && p.cache.width <= 128 && T * G * H >= 256 * 4 * kCus ? 8 : 4;
        const int64_t tile_rows = 32 * n.tile_waves;
        n.tile_tiles = T * G / tile_rows + p.seqs.seqs;     // see the kernel's numbering
        // those that have work, as far as the host can tell
        n.tile_splits = (int)splits_for(std::max<int64_t>(1, T * G / tile_rows) * H, kTileBlocks,
                                        std::min(len, seen + tile_rows / G + 1), kTilePart);
        if (n.tile_tiles * H * n.tile_splits > kMostBlocks) n.tile_splits = 1;
        part(T * p.q_heads, n.tile_splits, n.tile_o, n.tile_ml);
    }
    return n;
}

int check_attention(const echo_attention_args* p)
{
    if (!p) return ECHO_EINVAL;
    int rc = check_cache(p->cache);
    if (rc) return rc;
    if ((rc = check_seqs(p->seqs))) return rc;
    if (p->q_heads < 1 || p->q_heads % p->cache.heads || p->q_heads > kMaxRows) return ECHO_ESHAPE;
    if (p->seqs.tokens * p->q_heads > kMaxQueries || p->seqs.seqs * p->cache.heads > kMostBlocks) return ECHO_ESHAPE;
    const int64_t row = p->q_heads * p->cache.width;
    if (bad_ld(p->ld_q, p->seqs.tokens, row) || bad_ld(p->ld_out, p->seqs.tokens, row)) return ECHO_ESHAPE;
    if (p->window < 0 || (p->causal != 0 && p->causal != 1) || !std::isfinite(p->scale)) return ECHO_EINVAL;
    return ECHO_OK;
}

template <int KIND, int DP>
void attention_go(echo::AttnArgs& a, const AttnPlan& n, bool page16, hipStream_t st)
{
    const int64_t pairs = (int64_t)a.s.seqs * a.c.heads;
    if (n.tile) {
        a.tiles = (uint32_t)n.tile_tiles;
        const dim3 grid((unsigned)(n.tile_tiles * a.c.heads * n.tile_splits)), block(64 * n.tile_waves);
        if (!page16) {
            hipLaunchKernelGGL((echo::attention_tile_kernel<KIND, DP, 4, false>), grid, block, 0, st, a);
        } else if (n.tile_waves == 4) {
            hipLaunchKernelGGL((echo::attention_tile_kernel<KIND, DP, 4, true>), grid, block, 0, st, a);
        } else if constexpr (DP < 256) {
            hipLaunchKernelGGL((echo::attention_tile_kernel<KIND, DP, 8, true>), grid, block, 0, st, a);
        }
    }
    if (n.few) {
        a.tiles = (uint32_t)n.few_tiles;
        const dim3 grid((unsigned)(n.few_tiles * ceil_div(pairs * n.few_splits, 8) * 8)), block(64 * echo::kFewAttnWaves);
        if (page16) hipLaunchKernelGGL((echo::attention_few_kernel<KIND, DP, true>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((echo::attention_few_kernel<KIND, DP, false>), grid, block, 0, st, a);
    }
}

void attention_join(const echo::AttnArgs& a, int64_t rows, hipStream_t st)
{
    const dim3 grid(grid_of((rows + 3) / 4)), block(echo::kBlock);
    if (a.c.width <= 128) hipLaunchKernelGGL((echo::attention_join_kernel<128>), grid, block, 0, st, a, rows);
    else hipLaunchKernelGGL((echo::attention_join_kernel<256>), grid, block, 0, st, a, rows);
}

template <int KIND>
void attention_sized(echo::AttnArgs& a, const AttnPlan& n, bool page16, hipStream_t st)
{
    if (a.c.width <= 64) attention_go<KIND, 64>(a, n, page16, st);
    else if (a.c.width <= 128) attention_go<KIND, 128>(a, n, page16, st);
    else attention_go<KIND, 256>(a, n, page16, st);
}

}  // namespace

extern "C" {

int echo_cache_write(const echo_cache* cache, const echo_seqs* seqs, const void* k, int64_t ld_k, const void* v,
                     int64_t ld_v, int dtype, void* stream)
{
    return cache_io<true>(cache, seqs, (void*)k, ld_k, (void*)v, ld_v, dtype, stream);
}

int echo_cache_read(const echo_cache* cache, const echo_seqs* seqs, void* k, int64_t ld_k, void* v, int64_t ld_v,
                    int dtype, void* stream)
{
    return cache_io<false>(cache, seqs, k, ld_k, v, ld_v, dtype, stream);
}

size_t echo_cache_attention_workspace_bytes(const echo_attention_args* p)
{
    if (check_attention(p) || no_work(p->seqs)) return 0;
    return attn_plan(*p).total;
}

int echo_cache_attention(const echo_attention_args* p, void* workspace, size_t workspace_bytes, void* stream)
{
    int rc = check_attention(p);
    if (rc || no_work(p->seqs)) return rc;
    if ((rc = check_pointers(p->cache, p->seqs))) return rc;
    if (!p->q || !p->out) return ECHO_EINVAL;
    if (!aligned_to(p->q, 2) || !aligned_to(p->out, 2) || !aligned_to(p->lse, 4)) return ECHO_EALIGN;
    const AttnPlan plan = attn_plan(*p);
    if (plan.total && (!workspace || workspace_bytes < plan.total)) return ECHO_EINVAL;
    if (!aligned16(workspace)) return ECHO_EALIGN;
    echo::AttnArgs a;
    std::memset(&a, 0, sizeof(a));
    a.c = cache_view(p->cache);
    a.s = seq_view(p->seqs, p->cache);
    a.q = p->q; a.out = p->out; a.lse = p->lse; a.ld_q = p->ld_q; a.ld_out = p->ld_out;
    a.window = (int)std::min(p->window, kMaxRows); a.group = (int)(p->q_heads / p->cache.heads); a.causal = p->causal;
    a.scale2 = (float)((double)p->scale * 1.4426950408889634);
    uint8_t* ws = (uint8_t*)workspace;
    a.few_rows = plan.few && plan.tile ? (int)kFewBeside : 0;
    a.few = {plan.few_splits, (float*)ws, (float*)(ws + plan.few_ml)};
    a.tile = {plan.tile_splits, (float*)(ws + plan.tile_o), (float*)(ws + plan.tile_ml)};
    const hipStream_t st = (hipStream_t)stream;
    switch (p->cache.kind) {
    case ECHO_BF16: attention_sized<echo::kCacheBf16>(a, plan, paged16(p->cache), st); break;
    case ECHO_I8: attention_sized<echo::kCacheI8>(a, plan, paged16(p->cache), st); break;
    default: attention_sized<echo::kCacheI4>(a, plan, paged16(p->cache), st); break;
    }
    if ((rc = check_launch()) || !plan.total) return rc;
    attention_join(a, p->seqs.tokens * p->q_heads, st);
    return check_launch();
}

}  // extern "C"
