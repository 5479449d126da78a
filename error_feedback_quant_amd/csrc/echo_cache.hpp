// echo_cache.hpp — gfx950 kernels that quantize new keys and values into the
// paged cache and read them back, and what every kernel over the cache needs
// of its layout.
//
// A row (one token's elements of one head) is the quantization group: 8 bits
// by the token quantizer (a = max |u|, s = a / 127, q = rint(u * (127 / a))),
// 4 bits by the zero-aware quantizer with a binary16 scale and zero point.
#pragma once

#include "echo_int4.hpp"

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

// Sequence of row t, -1 where it is none's (or its sequence's rows leave those
// that there are): the last start at or below t.
// The starts are on the device, so the host cannot give a map; a search of
// log2(seqs) steps in L2 costs less than another launch.
__device__ __forceinline__ int seq_of_row(const SeqView& s, int64_t t)
{
    int lo = 0, hi = s.seqs;                    // the first start above t among 1 .. seqs is at lo + 1
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s.starts[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    const bool takes = lo < s.seqs && s.starts[lo] >= 0 && s.starts[lo] <= t && s.starts[lo + 1] <= s.tokens;
    return takes ? lo : -1;
}

struct CachePlace {
    bool none;              // of no sequence
    int32_t page;           // -1: no place
    uint32_t slot;
};

__device__ __forceinline__ CachePlace place_of_row(const SeqView& s, const CacheView& c, int64_t t)
{
    const int b = seq_of_row(s, t);
    if (b < 0) return {true, -1, 0};
    const int64_t pos = (int64_t)s.lens[b] - s.starts[b + 1] + t;
    if (pos < 0 || pos >= s.capacity) return {false, -1, 0};
    const uint32_t entry = (uint32_t)pos / c.page_tokens;          // capacity is below 2^32
    return {false, cache_page(s, c, b, entry), (uint32_t)pos - entry * c.page_tokens};
}

struct CacheIoArgs {
    CacheView c;
    SeqView s;
    void* x[2];             // new keys and values, or where they go
    int64_t ld[2];
    int64_t rows;           // tokens * heads, below 2^31
};

// L lanes share a row, 8 elements each; blockIdx.y 0 takes the keys, 1 the
// values.  Both kernels are one pass over memory.
template <int KIND, int L, bool BF16>
__global__ __launch_bounds__(kBlock) void cache_write_kernel(const CacheIoArgs a)
{
    constexpr uint32_t kRows = kBlock / L;
    const CacheView& c = a.c;
    const int part = blockIdx.y, g = threadIdx.x % L, k = 8 * g;
    uint8_t* codes = part ? c.v : c.k;
    uint32_t* scales = part ? c.vs : c.ks;
    for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < a.rows; r0 += (int64_t)gridDim.x * kRows) {
        const int64_t row = r0 + threadIdx.x / L;
        const bool in = row < a.rows;
        const uint32_t t = in ? (uint32_t)row / (uint32_t)c.heads : 0, h = in ? (uint32_t)row - t * (uint32_t)c.heads : 0;
        const Raw8<BF16> raw = ld_raw8<BF16, false>(a.x[part], (int64_t)t * a.ld[part] + (int64_t)h * c.width, k,
                                                    in ? c.width : 0);
        CachePlace p = place_of_row(a.s, c, t);
        const bool put = in && p.page >= 0;
        const int64_t at = p.page * c.ld_page + (int64_t)h * c.ld_head + (int64_t)p.slot * c.ld_token + k;
        const int64_t sat = p.page * c.ld_sp + (int64_t)h * c.ld_sh + p.slot;
        float u[8];
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            u[e] = raw_get(raw, e);
            top = max(top, abs_bits(u[e]));
        }
        if constexpr (KIND == kCacheBf16) {
            if (put && k < c.width) {
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = u[e];
                if constexpr (BF16) __builtin_memcpy(codes + 2 * at, raw.v, 16);
                else st_row8<true, false>(codes, at, 0, 8, o);
            }
        } else if constexpr (KIND == kCacheI8) {
            const TokenScale s = token_scale(group_max_u32<L>(top));
            int q[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] = token_code(u[e], s.inv);
            if (put && k < c.width) st_codes8<false>((int8_t*)codes, at, 0, 8, q);
            if (put && g == 0) scales[sat] = __builtin_bit_cast(uint32_t, s.scale);
        } else {
            uint32_t word;
            const uint32_t q = quantize4<L>(u, top, word);
            if (put && k < c.width) *(uint32_t*)(codes + at / 2) = q;
            if (put && g == 0) scales[sat] = word;
        }
    }
}

template <int KIND, int L, bool BF16>
__global__ __launch_bounds__(kBlock) void cache_read_kernel(const CacheIoArgs a)
{
    constexpr uint32_t kRows = kBlock / L;
    const CacheView& c = a.c;
    const int part = blockIdx.y, g = threadIdx.x % L, k = 8 * g;
    const uint8_t* codes = part ? c.v : c.k;
    const uint32_t* scales = part ? c.vs : c.ks;
    for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < a.rows; r0 += (int64_t)gridDim.x * kRows) {
        const int64_t row = r0 + threadIdx.x / L;
        if (row >= a.rows || k >= c.width) continue;
        const uint32_t t = (uint32_t)row / (uint32_t)c.heads, h = (uint32_t)row - t * (uint32_t)c.heads;
        const CachePlace p = place_of_row(a.s, c, t);
        if (p.none) continue;
        const int64_t to = (int64_t)t * a.ld[part] + (int64_t)h * c.width;
        float v[8];
        if (p.page < 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __builtin_bit_cast(float, 0x7FC00000u);
        } else {
            const int64_t at = p.page * c.ld_page + (int64_t)h * c.ld_head + (int64_t)p.slot * c.ld_token + k;
            const uint32_t word = KIND == kCacheBf16 ? 0u : scales[p.page * c.ld_sp + (int64_t)h * c.ld_sh + p.slot];
            if constexpr (KIND == kCacheBf16) {
                unpack_bf16x8(*(const u32x4*)(codes + 2 * at), v);
            } else if constexpr (KIND == kCacheI8) {
                const u32x2 w = *(const u32x2*)(codes + at);
                const float s = __builtin_bit_cast(float, word);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = (float)(int8_t)((e < 4 ? w.x : w.y) >> (8 * (e & 3))) * s;
            } else {
                const uint32_t w = *(const uint32_t*)(codes + at / 2);
                const float s = half_lo(word), z = half_hi(word);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = ((float)((w >> (4 * e)) & 15u) - z) * s;
            }
        }
        st_row8<BF16, false>(a.x[part], to, k, c.width, v);
    }
}

}  // namespace echo
