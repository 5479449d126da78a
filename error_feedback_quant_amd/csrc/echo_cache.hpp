// echo_cache.hpp — gfx950 kernels that quantize new keys and values into the
// paged cache and read them back, and what every kernel over the cache needs
// of its layout.
//
// A row (one token's elements of one head) is the quantization group: 8 bits
// by the token quantizer (a = max |u|, s = a / 127, q = rint(u * (127 / a))),
// 4 bits by the zero-aware quantizer with a binary16 scale and zero point.
#pragma once

#include "echo_int4.hpp"
#include "echo_search.hpp"

namespace echo {

enum CacheKind { kCacheBf16 = 1, kCacheI8 = 2, kCacheI4 = 3 };   // ECHO_BF16, ECHO_I8, ECHO_I4

struct CacheView {
    uint8_t* k;
    uint8_t* v;
    uint32_t* ks;           // fp32 scales or parameter words
    uint32_t* vs;
    int64_t ld_page, ld_head, ld_token, ld_sp, ld_sh;
    uint32_t pages, page_tokens;
    int heads, width;
};

struct SeqView {
    const int32_t* starts;
    const int32_t* lens;
    const int32_t* table;
    int64_t ld_table, table_pages;
    int64_t capacity;       // tokens that the table has entries for
    int seqs;
    int64_t tokens;
};

// bytes of n elements of a kind
template <int KIND>
__device__ __forceinline__ int64_t cache_bytes(int64_t n)
{
    return KIND == kCacheBf16 ? 2 * n : (KIND == kCacheI8 ? n : n / 2);
}

// Page that holds position t of sequence b; -1 where it has no place.
__device__ __forceinline__ int32_t cache_page(const SeqView& s, const CacheView& c, int b, uint32_t entry)
{
    const int32_t p = s.table[(int64_t)b * s.ld_table + entry];
    return (uint32_t)p < c.pages ? p : -1;
}

// The last i of 0 .. n - 1 with f(i) <= v (f does not decrease; 0 where there
// is none), for a v that the wave shares: 64 places at a time, so that it
// costs one trip to the cache up to 64 sequences and two up to 4096.
template <typename F>
__device__ __forceinline__ int last_at_most(int n, int64_t v, F f)
{
    WaveSearch s((uint32_t)n);
    while (s.turn()) {
        const uint32_t at = s.place(threadIdx.x & 63u);
        s.narrow(__popcll(__ballot(at < s.hi && f((int)at) <= v)));
    }
    return __builtin_amdgcn_readfirstlane((int)s.lo);
}

// whether row t is sequence b's and b is a sequence that is taken
__device__ __forceinline__ bool takes_row(const SeqView& s, int b, int64_t t)
{
    return s.starts[b] >= 0 && s.starts[b] <= t && s.starts[b + 1] > t && s.starts[b + 1] <= s.tokens;
}

// Sequence of row t, -1 where it is none's (or its sequence's rows leave those
// that there are).  from: the last one that starts at or below a row of the
// wave that is not behind t.
__device__ __forceinline__ int seq_of_row(const SeqView& s, int64_t t, int from)
{
    int lo = from;
    for (int i = 0; i < 4 && lo + 1 < s.seqs && s.starts[lo + 1] <= t; ++i) ++lo;    // the next ones, as in a decode step
    if (lo + 1 < s.seqs && s.starts[lo + 1] <= t) {
        int hi = s.seqs - 1;
        while (lo < hi) {
            const int mid = lo + (hi - lo + 1) / 2;
            if (s.starts[mid] <= t) lo = mid;
            else hi = mid - 1;
        }
    }
    return takes_row(s, lo, t) ? lo : -1;
}

struct CacheIoArgs {
    CacheView c;
    SeqView s;
    void* x[2];             // new keys and values, or where they go
    int64_t ld[2];
    int64_t rows;           // tokens * heads, below 2^31
};

// A wave's rows.  L lanes share a row, 8 elements each, so a pass takes 64 / L
// rows and U passes follow each other with all their loads on their way.
// Where a row lies takes two divisions, the sequence's numbers, its page and
// 64-bit products, which would bound the kernels: each lane finds out about one
// row and the others get its answer (30318 tokens x 8 x 128 from 8 bits: 92 us
// with every lane for itself, 42 us so).
template <int L, int U>
struct IoRows {
    static constexpr int kPass = 64 / L, kRows = kPass * U;
    static_assert(kRows <= 64, "a lane to a row");
    int64_t code, scale, x[2];      // of this lane's row; code -1: no place
    bool none;                      // no row, or no sequence's
    __device__ __forceinline__ IoRows(const CacheIoArgs& a)
    {
        const CacheView& c = a.c;
        const int64_t wave = (int64_t)blockIdx.x * (kBlock / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int64_t first = wave * kRows, row = first + (threadIdx.x & 63u);
        none = row >= a.rows || (threadIdx.x & 63u) >= (uint32_t)kRows;
        code = -1;
        scale = x[0] = x[1] = 0;
        const uint32_t t0 = (uint32_t)min(first, a.rows - 1) / (uint32_t)c.heads;
        const int from = last_at_most(a.s.seqs, t0, [&](int b) { return (int64_t)a.s.starts[b]; });
        if (none) return;
        const uint32_t t = (uint32_t)row / (uint32_t)c.heads, h = (uint32_t)row - t * (uint32_t)c.heads;
        const int b = seq_of_row(a.s, t, from);
        if (b < 0) {
            none = true;
            return;
        }
        x[0] = t * a.ld[0] + (int64_t)h * c.width;
        x[1] = t * a.ld[1] + (int64_t)h * c.width;
        const int64_t pos = (int64_t)a.s.lens[b] - a.s.starts[b + 1] + t;
        if (pos < 0 || pos >= a.s.capacity) return;
        const uint32_t entry = (uint32_t)pos / c.page_tokens, slot = (uint32_t)pos - entry * c.page_tokens;
        const int32_t page = cache_page(a.s, c, b, entry);
        if (page < 0) return;
        code = page * c.ld_page + h * c.ld_head + slot * c.ld_token;
        scale = page * c.ld_sp + h * c.ld_sh + slot;
    }
    // of the row that this lane has a share in, in pass u
    struct Row {
        int64_t code, scale, x;
        bool none;
    };
    __device__ __forceinline__ Row of(int u, int part) const
    {
        const int from = u * kPass + (threadIdx.x & 63u) / L;
        return {__shfl(code, from), __shfl(scale, from), __shfl(part ? x[1] : x[0], from), __shfl((int)none, from) != 0};
    }
};

template <int KIND, int L, int U, bool BF16>
__global__ __launch_bounds__(kBlock) void cache_write_kernel(const CacheIoArgs a)
{
    const CacheView& c = a.c;
    const int part = blockIdx.y, g = threadIdx.x % L, k = 8 * g;
    uint8_t* codes = part ? c.v : c.k;
    uint32_t* scales = part ? c.vs : c.ks;
    const IoRows<L, U> rows(a);
    typename IoRows<L, U>::Row r[U];
    Raw8<BF16> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        r[u] = rows.of(u, part);
        raw[u] = ld_raw8<BF16, false>(a.x[part], r[u].x, k, r[u].none ? 0 : c.width);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const bool put = r[u].code >= 0, mine = put && k < c.width;
        const int64_t at = r[u].code + k;
        float v[8];
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e] = raw_get(raw[u], e);
            top = max(top, abs_bits(v[e]));
        }
        if constexpr (KIND == kCacheBf16) {
            if (mine) {
                if constexpr (BF16) __builtin_memcpy(codes + 2 * at, raw[u].v, 16);
                else st_row8<true, false>(codes, at, 0, 8, v);
            }
        } else if constexpr (KIND == kCacheI8) {
            const TokenScale s = token_scale(group_max_u32<L>(top));
            int q[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] = token_code(v[e], s.inv);
            if (mine) st_codes8<false>((int8_t*)codes, at, 0, 8, q);
            if (put && g == 0) scales[r[u].scale] = __builtin_bit_cast(uint32_t, s.scale);
        } else {
            uint32_t word;
            const uint32_t q = quantize4<L>(v, top, word);
            if (mine) *(uint32_t*)(codes + at / 2) = q;
            if (put && g == 0) scales[r[u].scale] = word;
        }
    }
}

template <int KIND, int L, int U, bool BF16>
__global__ __launch_bounds__(kBlock) void cache_read_kernel(const CacheIoArgs a)
{
    const CacheView& c = a.c;
    const int part = blockIdx.y, g = threadIdx.x % L, k = 8 * g;
    const uint8_t* codes = part ? c.v : c.k;
    const uint32_t* scales = part ? c.vs : c.ks;
    const IoRows<L, U> rows(a);
    typename IoRows<L, U>::Row r[U];
    constexpr int kWords = KIND == kCacheBf16 ? 4 : (KIND == kCacheI8 ? 2 : 1);
    uint32_t w[U][kWords], word[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        r[u] = rows.of(u, part);
        const bool get = r[u].code >= 0 && k < c.width;
        word[u] = get && KIND != kCacheBf16 ? scales[r[u].scale] : 0u;
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[u][i] = 0;
        if (get) __builtin_memcpy(w[u], __builtin_assume_aligned(codes + cache_bytes<KIND>(r[u].code + k), 4 * kWords), 4 * kWords);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (r[u].none || k >= c.width) continue;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (KIND == kCacheBf16) v[e] = e & 1 ? bf16_hi(w[u][e / 2]) : bf16_lo(w[u][e / 2]);
            else if constexpr (KIND == kCacheI8) v[e] = (float)(int8_t)(w[u][e / 4] >> (8 * (e & 3))) * __builtin_bit_cast(float, word[u]);
            else v[e] = ((float)((w[u][0] >> (4 * e)) & 15u) - half_hi(word[u])) * half_lo(word[u]);
            if (r[u].code < 0) v[e] = __builtin_bit_cast(float, 0x7FC00000u);
        }
        st_row8<BF16, false>(a.x[part], r[u].x, k, c.width, v);
    }
}

}  // namespace echo
