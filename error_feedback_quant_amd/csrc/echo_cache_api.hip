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

template <int KIND, int L, bool WRITE>
void cache_io_go(const echo::CacheIoArgs& a, bool bf16, hipStream_t st)
{
    const int64_t rows = echo::kBlock / L;
    const dim3 grid(grid_of((a.rows + rows - 1) / rows), 2), block(echo::kBlock);
    if constexpr (WRITE) {
        if (bf16) hipLaunchKernelGGL((echo::cache_write_kernel<KIND, L, true>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((echo::cache_write_kernel<KIND, L, false>), grid, block, 0, st, a);
    } else {
        if (bf16) hipLaunchKernelGGL((echo::cache_read_kernel<KIND, L, true>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((echo::cache_read_kernel<KIND, L, false>), grid, block, 0, st, a);
    }
}

template <int KIND, bool WRITE>
void cache_io_sized(const echo::CacheIoArgs& a, bool bf16, hipStream_t st)
{
    if (a.c.width <= 64) cache_io_go<KIND, 8, WRITE>(a, bf16, st);
    else if (a.c.width <= 128) cache_io_go<KIND, 16, WRITE>(a, bf16, st);
    else cache_io_go<KIND, 32, WRITE>(a, bf16, st);
}

template <bool WRITE>
int cache_io(const echo_cache* c, const echo_seqs* s, void* k, int64_t ld_k, void* v, int64_t ld_v, int dtype, void* stream)
{
    if (!c || !s) return ECHO_EINVAL;
    if (!float_dtype(dtype)) return ECHO_EUNSUP;
    int rc = check_cache(*c);
    if (rc) return rc;
    if ((rc = check_seqs(*s))) return rc;
    if (s->tokens * c->heads > kMaxRows || bad_ld(ld_k, s->tokens, c->heads * c->width) ||
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
    int64_t tile_tiles;     // row tiles of all sequences together, at most
    int splits;             // parts of a row's tokens
    size_t part_ml, total;  // of the workspace: the parts' sums of v, then their m and l
};

#ifndef TW
#define TW 4
#endif
constexpr int kTileWaves = TW;
constexpr int64_t kTileRows = 32 * kTileWaves;
constexpr int64_t kFewBlocks = 4 * kCus, kFewPart = 256, kTileBlocks = 2 * kCus, kTilePart = 512, kMostSplits = 256;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

AttnPlan attn_plan(const echo_attention_args& p)
{
    AttnPlan n = {};
    const int64_t G = p.q_heads / p.cache.heads, T = p.seqs.tokens, pairs = p.seqs.seqs * p.cache.heads;
    const int64_t most_new = std::max<int64_t>(1, std::min(p.seqs.max_new, T));
    n.tile = most_new * G > echo::kFewRows;
    n.few = !n.tile || p.seqs.seqs > 1;
    n.few_tiles = n.tile ? 1 : ceil_div(most_new * G, echo::kFewRows);
    n.tile_tiles = T * G / kTileRows + p.seqs.seqs;         // see the kernel's numbering
    // tokens that a row tile sees at most
    int64_t len = std::min(p.seqs.max_len, p.seqs.table_pages * p.cache.page_tokens);
    if (p.window > 0) len = std::min(len, std::min(p.window, len) + ceil_div(n.tile ? kTileRows : echo::kFewRows, G));
    // blocks that have work, as far as the host can tell
    const int64_t blocks = n.tile ? std::max<int64_t>(1, T * G / kTileRows) * p.cache.heads : n.few_tiles * pairs;
    int64_t splits = ceil_div(n.tile ? kTileBlocks : kFewBlocks, blocks);
    splits = std::min(splits, std::min(ceil_div(len, n.tile ? kTilePart : kFewPart), kMostSplits));
    // a launch's blocks are 32 bits: the kernels stride over the row tiles
    const int64_t most = std::max<int64_t>(1, (int64_t(1) << 24) / pairs);
    n.splits = (int)std::max<int64_t>(1, std::min(splits, most));
    n.few_tiles = std::max<int64_t>(1, std::min(n.few_tiles, most / n.splits));
    if (n.tile && n.tile_tiles * p.cache.heads * n.splits >= int64_t(1) << 24) n.splits = 1;
    if (n.splits > 1) {
        const int64_t rows = T * p.q_heads;
        n.part_ml = (size_t)(rows * n.splits * p.cache.width * 4);
        n.total = n.part_ml + (size_t)(rows * n.splits * 8);
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
    if (p->seqs.tokens * p->q_heads > kMaxRows || p->seqs.seqs * p->cache.heads > (int64_t(1) << 24)) return ECHO_ESHAPE;
    const int64_t row = p->q_heads * p->cache.width;
    if (bad_ld(p->ld_q, p->seqs.tokens, row) || bad_ld(p->ld_out, p->seqs.tokens, row)) return ECHO_ESHAPE;
    if (p->window < 0 || (p->causal != 0 && p->causal != 1) || !std::isfinite(p->scale)) return ECHO_EINVAL;
    return ECHO_OK;
}

template <int KIND, int DP>
void attention_go(echo::AttnArgs& a, const AttnPlan& n, hipStream_t st)
{
    // 16 tokens of a page at 32-bit offsets from the first
    const bool page16 = a.c.page_tokens % 16 == 0 && a.c.ld_token < int64_t(1) << 26;
    const int64_t pairs = (int64_t)a.s.seqs * a.c.heads * n.splits;
    a.few_rows = n.few && n.tile ? echo::kFewRows : 0;
    if (n.tile) {
        a.tiles = (uint32_t)n.tile_tiles;
        const dim3 grid((unsigned)(n.tile_tiles * a.c.heads * n.splits)), block(64 * kTileWaves);
        if (page16) hipLaunchKernelGGL((echo::attention_tile_kernel<KIND, DP, kTileWaves, 1, true>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((echo::attention_tile_kernel<KIND, DP, kTileWaves, 1, false>), grid, block, 0, st, a);
    }
    if (n.few) {
        a.tiles = (uint32_t)n.few_tiles;
        const dim3 grid((unsigned)(n.few_tiles * pairs)), block(64 * echo::kFewAttnWaves);
        if (page16) hipLaunchKernelGGL((echo::attention_few_kernel<KIND, DP, true>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((echo::attention_few_kernel<KIND, DP, false>), grid, block, 0, st, a);
    }
}

template <int KIND>
void attention_sized(echo::AttnArgs& a, const AttnPlan& n, hipStream_t st)
{
    if (a.c.width <= 64) attention_go<KIND, 64>(a, n, st);
    else if (a.c.width <= 128) attention_go<KIND, 128>(a, n, st);
    else attention_go<KIND, 256>(a, n, st);
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
    a.splits = plan.splits;
    a.part_o = (float*)workspace;
    a.part_ml = (float*)((uint8_t*)workspace + plan.part_ml);
    const hipStream_t st = (hipStream_t)stream;
    switch (p->cache.kind) {
    case ECHO_BF16: attention_sized<echo::kCacheBf16>(a, plan, st); break;
    case ECHO_I8: attention_sized<echo::kCacheI8>(a, plan, st); break;
    default: attention_sized<echo::kCacheI4>(a, plan, st); break;
    }
    if ((rc = check_launch()) || plan.splits == 1) return rc;
    const int64_t rows = p->seqs.tokens * p->q_heads;
    hipLaunchKernelGGL(echo::attention_join_kernel, dim3(grid_of((rows + 3) / 4)), dim3(echo::kBlock), 0, st, a, rows);
    return check_launch();
}

}  // extern "C"
