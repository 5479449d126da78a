// echo_attention.hpp — gfx950 kernels of attention over the paged cache.
//
// For a row (one query head of one new token) with scores x_j = scale q . k_j
// over the tokens it sees: out = sum_j 2^(y_j - m) v_j / sum_j 2^(y_j - m)
// with y = x log2(e) and any m; lse = ln 2 (m + log2 sum).  One pass over the
// cache keeps m, the sum l and the sum of v for every row; parts over
// different tokens join by scaling to the larger m.
//
// Codes stay codes up to the matrix cores.  With k_j = s_j (c_j - z_j) and
// v_j = t_j (d_j - w_j), a score is s_j (q . c_j - z_j sum q) and the output
// takes p_j t_j times d_j: 8-bit codes are exact in bfloat16, and 4-bit codes
// are 16 + c (echo_int4.hpp), whose offset is taken off the score through the
// sum of q and off the output through sum_j bf16(p_j t_j) (16 + w_j), one
// number a row.  p_j t_j is rounded to bfloat16 (half a unit of 2^-8), the
// type of the matrix operand; m, l and all sums are fp32.
//
// Both products take tokens as the rows (of k) or the depth (of v) of the
// first operand and query rows as the columns of the second, so a lane keeps
// one query row throughout: its scores, weights, m and l stay in its own
// registers from the first product to the second, where they are the second
// operand as they are.
//
// A masked token has weight 0, but 0 times an infinity or a NaN in v is NaN.
// Codes are finite, and a scale enters through p_j t_j, which a mask sets to
// 0.  In a bfloat16 cache the elements of v that are no numbers are set to 0
// where a tile is masked in part, and the rows that see their token get the
// weight NaN.
#pragma once

#include "echo_cache.hpp"

namespace echo {

struct AttnArgs {
    CacheView c;
    SeqView s;
    const uint16_t* q;
    uint16_t* out;
    float* lse;
    int64_t ld_q, ld_out;
    int window;             // 0: all
    int group;              // query heads of a head of the cache
    int causal;
    float scale2;           // scale * log2(e)
    int splits;             // parts of a row's tokens
    uint32_t tiles;         // row tiles of a sequence that have a block of their own
    int few_rows;           // rows up to which a sequence is the few-row kernel's, 0: the launched kernel takes all
    float* part_o;          // [rows][splits][width]
    float* part_ml;         // [rows][splits][2]
};

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRaise = 8.0f;   // a row's m follows its largest score when that is 2^8 above it

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float nan_f32() { return __builtin_bit_cast(float, 0x7FC00000u); }
__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// largest / sum over the four 16-lane rows of a wave (lanes that share lane % 16)
__device__ __forceinline__ float rows4_max(float v)
{
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float rows4_sum(float v)
{
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// What a block needs to know of its sequence.  Positions are 32 bits: the host
// keeps the capacity below 2^31 - 2^12, and a row before the first token
// stands at -1, which sees as little.
struct RowSpan {
    int row0;               // first row of the sequence
    int n, len;             // its rows and tokens
    __device__ __forceinline__ int pos(int i) const { return max(len - n + i, -1); }
};
__device__ __forceinline__ RowSpan seq_span(const SeqView& s, int b)
{
    RowSpan r;
    const int e = s.starts[b + 1];
    r.row0 = s.starts[b];
    r.len = max(s.lens[b], 0);
    r.n = r.row0 < 0 || e > s.tokens || e < r.row0 ? 0 : e - r.row0;
    return r;
}

// Tokens [begin, end) that any of rows i0 .. i1 of a sequence sees, as far as
// the table goes; begin a multiple of 32.
__device__ __forceinline__ void seen_span(const AttnArgs& a, const RowSpan& r, int i0, int i1, int& begin, int& end)
{
    end = min(a.causal ? r.pos(i1) + 1 : r.len, (int)a.s.capacity);
    begin = a.window ? max(r.pos(i0) - a.window + 1, 0) & ~31 : 0;
    end = max(end, begin);
}

// The part [begin, end) of one split: equal runs of a multiple of 128 tokens.
__device__ __forceinline__ void split_span(int splits, int split, int& begin, int& end)
{
    if (splits == 1) return;
    const int64_t per = (((int64_t)end - begin + splits - 1) / splits + 127) & ~(int64_t)127;
    const int64_t from = min(begin + split * per, (int64_t)end);
    end = (int)min(from + per, (int64_t)end);
    begin = (int)from;
}

// Out and lse of a row whose sums are whole; sees_past: it sees a token that
// the table has no entry for.
__device__ __forceinline__ float row_lse(float m, float l) { return (m + __builtin_log2f(l)) * kLn2; }

// -------------------------------------------------------------- few rows --
//
// Up to 16 rows (query heads that share a head of the cache, times new
// tokens) to a block of four waves; a wave takes every fourth tile of 32
// tokens of the block's part on its own, without barriers, and the waves'
// sums meet in LDS at the end.  Nothing else goes through LDS: a lane's loads
// of k are its operand, and of v it takes the same 8 elements of the 8 tokens
// that its 16-lane row stands for, so the transposition that the second
// product asks for is a choice of bytes between its own registers.

constexpr int kFewRows = 16;
constexpr int kFewTile = 32;
constexpr int kFewAttnWaves = 4;

template <int KIND, int DP>
struct FewShape {
    static constexpr int kE = KIND == kCacheBf16 ? 8 : (KIND == kCacheI8 ? 16 : (DP == 64 ? 16 : 32));   // of k, a load
    static constexpr int kLoads = DP / (4 * kE);                                                      // a token
    static constexpr int kKWords = KIND == kCacheBf16 ? 4 : (KIND == kCacheI8 ? 4 : kE / 8);
    static constexpr int kVE = DP == 64 ? 4 : 8;                                                      // of v, a piece
    static constexpr int kPieces = DP / (16 * kVE);
    static constexpr int kVBytes = KIND == kCacheBf16 ? 2 * kVE : (KIND == kCacheI8 ? kVE : kVE / 2);
    static constexpr int kVWords = (kVBytes + 3) / 4;
};

template <int KIND, int DP>
struct FewTile {
    using S = FewShape<KIND, DP>;
    uint32_t k[2][S::kLoads][S::kKWords];
    uint32_t v[8][S::kPieces][S::kVWords];
    uint32_t ks[8], vs[8];      // of the lane's 8 tokens
    uint32_t bad;               // its tokens without a place, by bits
};

// 8 elements of k (words) as bfloat16
template <int KIND>
__device__ __forceinline__ bf16x8 k_frag(const uint32_t* w)
{
    u32x4 o;
    if constexpr (KIND == kCacheBf16) {
        o = u32x4{w[0], w[1], w[2], w[3]};
    } else if constexpr (KIND == kCacheI8) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = upper_pair((float)(int8_t)(w[i / 2] >> (16 * (i & 1))), (float)(int8_t)(w[i / 2] >> (16 * (i & 1) + 8)));
    } else {
        return codes_bf16(w[0]);
    }
    return __builtin_bit_cast(bf16x8, o);
}

// element f of 8 tokens' pieces of v
template <int KIND, int WORDS>
__device__ __forceinline__ bf16x8 v_frag(const uint32_t (*v)[WORDS], int f)
{
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (KIND == kCacheBf16) {
            o[i] = __builtin_amdgcn_perm(v[2 * i + 1][f / 2], v[2 * i][f / 2], f & 1 ? 0x07060302u : 0x05040100u);
        } else if constexpr (KIND == kCacheI8) {
            o[i] = upper_pair((float)(int8_t)(v[2 * i][f / 4] >> (8 * (f & 3))),
                              (float)(int8_t)(v[2 * i + 1][f / 4] >> (8 * (f & 3))));
        } else {
            const uint32_t h = __builtin_amdgcn_perm(v[2 * i + 1][0], v[2 * i][0], f < 4 ? 0x05040100u : 0x07060302u);
            const int at = 4 * (f & 3);
            o[i] = ((at ? h >> (at - 3) : h << 3) & 0x00780078u) | 0x41804180u;
        }
    }
    return __builtin_bit_cast(bf16x8, o);
}

// Halves of a word that are no finite bfloat16, as a mask
__device__ __forceinline__ uint32_t not_finite2(uint32_t w)
{
    uint32_t m = (w & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u;
    return m | ((w & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
}

// PAGE16: pages are a multiple of 16 tokens, so the 16 tokens of a tile's half
// lie in one page; otherwise every lane looks its tokens up.
template <int KIND, int DP, bool PAGE16>
__global__ __launch_bounds__(64 * kFewAttnWaves) void attention_few_kernel(const AttnArgs a)
{
    using S = FewShape<KIND, DP>;
    constexpr int kFrags = S::kPieces * S::kVE;
    constexpr int kSteps = DP / 32;
    constexpr int kPitch = DP + 4;
    __shared__ float so[kFewAttnWaves][kFewRows][kPitch];
    __shared__ float sm[kFewAttnWaves][kFewRows], sl[kFewAttnWaves][kFewRows];
    const CacheView& c = a.c;
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, g = lane >> 4;
    uint32_t id = blockIdx.x;
    const int split = id % (uint32_t)a.splits;
    id /= (uint32_t)a.splits;
    const int h = id % (uint32_t)c.heads;
    id /= (uint32_t)c.heads;
    const int b = id % (uint32_t)a.s.seqs;
    const RowSpan r = seq_span(a.s, b);
    const int rows = r.n * a.group;                      // below 2^31 with all heads
    if (a.few_rows && rows > a.few_rows) return;         // the other kernel's
    const uint8_t* kb = c.k + cache_bytes<KIND>(h * c.ld_head);
    const uint8_t* vb = c.v + cache_bytes<KIND>(h * c.ld_head);

    for (int64_t rt = id / (uint32_t)a.s.seqs; rt * kFewRows < rows; rt += a.tiles) {
        // this lane's row
        const int64_t rr = rt * kFewRows + col;
        const bool there = rr < rows;
        const int i = there ? (int)rr / a.group : 0;
        const int64_t t = r.row0 + i;
        const int qh = h * a.group + (there ? (int)rr - i * a.group : 0);
        const int pos = r.pos(i);
        const int hi = there ? (a.causal ? pos : r.len - 1) : -1;              // it sees lo .. hi
        const int lo = a.window ? pos - a.window + 1 : 0;
        int begin, end;
        seen_span(a, r, (int)rt * kFewRows / a.group, ((int)min((int64_t)rows, (rt + 1) * kFewRows) - 1) / a.group, begin, end);
        split_span(a.splits, split, begin, end);

        // q as the second operand, in the order of k's elements
        bf16x8 fq[kSteps];
        float qsum = 0.0f;
#pragma unroll
        for (int st = 0; st < kSteps; ++st) {
            constexpr int kPer = S::kE / 8;
            const int d = S::kE * (4 * (st / kPer) + g) + 8 * (st % kPer);
            const Raw8<true> raw = ld_raw8<true, false>(a.q, t * a.ld_q + (int64_t)qh * c.width, d, c.width);
            if constexpr (KIND == kCacheI4) {
                bf16x8 f[1];
                x_parts<true, 1>(raw, f);
                fq[st] = f[0];
#pragma unroll
                for (int e = 0; e < 8; ++e) qsum += raw_get(raw, e);
            } else {
                fq[st] = __builtin_bit_cast(bf16x8, raw.v[0]);
            }
        }
        if constexpr (KIND == kCacheI4) qsum = rows4_sum(qsum);

        auto load = [&](FewTile<KIND, DP>& f, int p0) {
            // where the lane's tokens lie: of k two, of v (and the scores) 8
            int64_t ko[2], vo[8], sc[8];
            f.bad = 0;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if constexpr (PAGE16) {
                    const uint32_t p = (uint32_t)min(p0 + 16 * u, end - 1);
                    const uint32_t entry = p / c.page_tokens;
                    const int32_t page = __builtin_amdgcn_readfirstlane(cache_page(a.s, c, b, entry));
                    if (page < 0) f.bad |= 15u << (4 * u);
                    const int64_t pg = page < 0 ? 0 : page;
                    const uint32_t slot = (p - entry * c.page_tokens) & ~15u;
                    ko[u] = pg * c.ld_page + (int64_t)(slot + col) * c.ld_token;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        vo[4 * u + e] = pg * c.ld_page + (int64_t)(slot + 4 * g + e) * c.ld_token;
                        sc[4 * u + e] = pg * c.ld_sp + h * c.ld_sh + slot + 4 * g + e;
                    }
                } else {
                    auto place = [&](int at, int64_t& o, int64_t& s) {
                        const uint32_t p = (uint32_t)min(at, end - 1);
                        const uint32_t entry = p / c.page_tokens;
                        const int32_t page = cache_page(a.s, c, b, entry);
                        const int64_t pg = page < 0 ? 0 : page;
                        const uint32_t slot = p - entry * c.page_tokens;
                        o = pg * c.ld_page + (int64_t)slot * c.ld_token;
                        s = pg * c.ld_sp + h * c.ld_sh + slot;
                        return page < 0;
                    };
                    int64_t none;
                    place(p0 + 16 * u + col, ko[u], none);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (place(p0 + 16 * u + 4 * g + e, vo[4 * u + e], sc[4 * u + e])) f.bad |= 1u << (4 * u + e);
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int j = 0; j < S::kLoads; ++j) {
                    const int d = S::kE * (4 * j + g);
                    const uint8_t* from = kb + cache_bytes<KIND>(ko[u] + d);
                    if (d + S::kE <= c.width) {
                        __builtin_memcpy(f.k[u][j], __builtin_assume_aligned(from, 4), 4 * S::kKWords);
                    } else {                                 // q is 0 past the width, and so has k to be
                        constexpr int kWords8 = S::kKWords * 8 / S::kE;     // of 8 elements
#pragma unroll
                        for (int w = 0; w < S::kKWords; ++w)
                            f.k[u][j][w] = d + w / kWords8 * 8 < c.width ? ((const uint32_t*)from)[w] : 0u;
                    }
                }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
#pragma unroll
                for (int p = 0; p < S::kPieces; ++p) {
                    const int d = 128 * p + S::kVE * col;
#pragma unroll
                    for (int w = 0; w < S::kVWords; ++w) f.v[e][p][w] = 0;
                    if (d < c.width) __builtin_memcpy(f.v[e][p], vb + cache_bytes<KIND>(vo[e] + d), S::kVBytes);
                }
                if constexpr (KIND != kCacheBf16) {
                    f.ks[e] = c.ks[sc[e]];
                    f.vs[e] = c.vs[sc[e]];
                }
            }
        };

        f32x4 o[kFrags];
#pragma unroll
        for (int f = 0; f < kFrags; ++f) o[f] = f32x4{0, 0, 0, 0};
        float m = neg_inf(), l = 0.0f, off = 0.0f;           // off: what the codes' offsets add to every element

        auto take = [&](FewTile<KIND, DP>& f, int p0) {
            f32x4 acc[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                acc[u] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int st = 0; st < kSteps; ++st) {
                    constexpr int kPer = S::kE / 8, kW = S::kKWords / kPer;
                    acc[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k_frag<KIND>(&f.k[u][st / kPer][kW * (st % kPer)]),
                                                                     fq[st], acc[u], 0, 0, 0);
                }
            }
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float s = acc[e / 4][e % 4];
                if constexpr (KIND == kCacheBf16) x[e] = s * a.scale2;
                else if constexpr (KIND == kCacheI8) x[e] = s * (__builtin_bit_cast(float, f.ks[e]) * a.scale2);
                else x[e] = __builtin_fmaf(-(16.0f + half_hi(f.ks[e])), qsum, s) * (half_lo(f.ks[e]) * a.scale2);
            }
            // which of the tile's tokens the row sees
            const bool whole = __all(!there || (lo <= p0 && p0 + kFewTile - 1 <= hi)) && p0 + kFewTile <= end;
            uint32_t odd = 0, seen = 255;                    // tokens whose v holds no number; that the row sees
            const bool bad = __any(f.bad != 0);
            if (!whole || bad) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int p = p0 + 16 * (e / 4) + 4 * g + (e & 3);
                    const bool sees = p >= lo && p <= hi && p < end;
                    if ((f.bad >> e) & 1u) x[e] = nan_f32();
                    if (!sees) {
                        x[e] = neg_inf();
                        seen &= ~(1u << e);
                    }
                }
                if constexpr (KIND == kCacheBf16) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
#pragma unroll
                        for (int p = 0; p < S::kPieces; ++p)
#pragma unroll
                            for (int w = 0; w < S::kVWords; ++w) {
                                const uint32_t no = not_finite2(f.v[e][p][w]);
                                f.v[e][p][w] &= ~no;
                                odd |= no ? 1u << e : 0u;
                            }
                    odd = group_fold<16>(odd, [](uint32_t p, uint32_t q) { return p | q; });
                }
            }
            float top = x[0];
#pragma unroll
            for (int e = 1; e < 8; ++e) top = fmaxf(top, x[e]);
            if (__any(top > m + kRaise)) {
                // row by row, so that no row's rounding goes by another's scores
                top = rows4_max(top);
                const float up = top > m + kRaise ? top : m;
                const float fac = up == m ? 1.0f : exp2_fast(m - up);
                m = up;
                l *= fac;
                off *= fac;
#pragma unroll
                for (int j = 0; j < kFrags; ++j) o[j] *= fac;
            }
            const float base = m == neg_inf() ? 0.0f : m;
            float p[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                p[e] = exp2_fast(x[e] - base);
                l += p[e];
                const bool sees = (seen >> e) & 1u;
                if constexpr (KIND == kCacheI8) p[e] = sees ? p[e] * __builtin_bit_cast(float, f.vs[e]) : 0.0f;
                if constexpr (KIND == kCacheI4) p[e] = sees ? p[e] * half_lo(f.vs[e]) : 0.0f;
                if (KIND == kCacheBf16 && sees && ((odd >> e) & 1u)) p[e] = nan_f32();
            }
            bf16x8 fp;
#pragma unroll
            for (int e = 0; e < 8; ++e) fp[e] = (__bf16)p[e];
            if constexpr (KIND == kCacheI4) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if ((seen >> e) & 1u) off = __builtin_fmaf((float)fp[e], 16.0f + half_hi(f.vs[e]), off);
            }
#pragma unroll
            for (int pc = 0; pc < S::kPieces; ++pc) {
                uint32_t v[8][S::kVWords];
#pragma unroll
                for (int e = 0; e < 8; ++e)
#pragma unroll
                    for (int w = 0; w < S::kVWords; ++w) v[e][w] = f.v[e][pc][w];
#pragma unroll
                for (int j = 0; j < S::kVE; ++j)
                    o[S::kVE * pc + j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v_frag<KIND, S::kVWords>(v, j), fp,
                                                                               o[S::kVE * pc + j], 0, 0, 0);
            }
        };
        for (int p0 = begin + kFewTile * (int)wave; p0 < end; p0 += kFewTile * kFewAttnWaves) {
            FewTile<KIND, DP> f;
            load(f, p0);
            take(f, p0);
        }

        // the waves' sums to the largest m
        l = rows4_sum(l);
        if constexpr (KIND == kCacheI4) off = rows4_sum(off);
        if (g == 0) {
            sm[wave][col] = m;
            sl[wave][col] = l;
        }
        __syncthreads();
        float top = sm[0][col];
#pragma unroll
        for (int w = 1; w < kFewAttnWaves; ++w) top = fmaxf(top, sm[w][col]);
        const float fac = m == neg_inf() ? (l == 0.0f ? 0.0f : l) : exp2_fast(m - top);   // m of -inf: l is 0 or NaN
#pragma unroll
        for (int pc = 0; pc < S::kPieces; ++pc)
#pragma unroll
            for (int v = 0; v < 4; ++v)
#pragma unroll
                for (int j = 0; j < S::kVE; j += 4) {
                    f32x4 w;
#pragma unroll
                    for (int k = 0; k < 4; ++k) w[k] = (o[S::kVE * pc + j + k][v] - off) * fac;
                    *(f32x4*)&so[wave][col][128 * pc + S::kVE * (4 * g + v) + j] = w;
                }
        __syncthreads();
        // 8 elements of a row to a thread
        for (uint32_t u = tid; u < kFewRows * (DP / 8); u += 64 * kFewAttnWaves) {
            const int q = u / (DP / 8), d = 8 * (u % (DP / 8));
            const int64_t row = rt * kFewRows + q;
            if (row >= rows || d >= c.width) continue;
            float mm = sm[0][q];
#pragma unroll
            for (int w = 1; w < kFewAttnWaves; ++w) mm = fmaxf(mm, sm[w][q]);
            float ll = 0.0f, e[8] = {};
#pragma unroll
            for (int w = 0; w < kFewAttnWaves; ++w) {
                ll += sm[w][q] == neg_inf() ? sl[w][q] : sl[w][q] * exp2_fast(sm[w][q] - mm);
#pragma unroll
                for (int k = 0; k < 8; ++k) e[k] += so[w][q][d + k];
            }
            const int i2 = (int)row / a.group;
            const int64_t t2 = r.row0 + i2;
            const int64_t at = t2 * c.heads * a.group + h * a.group + (row - i2 * a.group);
            const int last = a.causal ? r.pos(i2) : r.len - 1;
            if (last >= a.s.capacity) ll = nan_f32();        // it sees tokens that the table does not hold
            if (a.splits > 1) {
                float* po = a.part_o + (at * a.splits + split) * c.width + d;
                *(f32x4*)po = f32x4{e[0], e[1], e[2], e[3]};
                *(f32x4*)(po + 4) = f32x4{e[4], e[5], e[6], e[7]};
                if (d == 0) *(f32x2*)(a.part_ml + 2 * (at * a.splits + split)) = f32x2{mm, ll};
            } else {
                const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
#pragma unroll
                for (int k = 0; k < 8; ++k) e[k] *= inv;
                st_row8<true, false>(a.out, t2 * a.ld_out + (int64_t)(h * a.group + (row - i2 * a.group)) * c.width, d, c.width, e);
                if (d == 0 && a.lse) a.lse[at] = row_lse(mm, ll);
            }
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------- many rows --
//
// A block of four waves takes 128 QR rows of one sequence and head of the
// cache, 32 QR to a wave, and walks over the tokens in tiles of 8192 / DP.  A
// tile is loaded into registers while the one before it is multiplied, turned
// into bfloat16 and laid into one of two stages of LDS, in the order of the
// matrix operands: every read of a fragment is 64 consecutive 16-byte words.
//
// A thread stages 8 tokens by 8 elements, of k or of v.  Of v it writes, for
// each of its elements, the 8 tokens: the transposition costs the byte
// permutations that the change of type needs anyway.  Tokens and elements of
// the fragments of v are permuted so that the weights leave the first product
// as the second one's operand, and so that the writes of 16 lanes fall on
// consecutive words; k's words are spread by an exclusive or.

template <int DP>
struct TileShape {
    static constexpr int kTokens = 8192 / DP;            // of a tile
    static constexpr int kUnits = DP / 8;                // of 8 elements
    static constexpr int kSubs = kTokens / 32;           // 32 tokens: the rows of a first product
    static constexpr int kSteps = kTokens / 16;          // 16 tokens: the depth of a second one
    static constexpr int kParts = DP / 32;               // 32 elements: the rows of a second one
    static constexpr int kEach = 32 / kUnits;            // elements of a unit in a part
};

constexpr int kTileWaves = 4;

template <int KIND>
struct RawUnit {                                         // 8 elements as they lie in the cache
    uint32_t w[KIND == kCacheBf16 ? 4 : (KIND == kCacheI8 ? 2 : 1)];
};

// element e of a unit as a float that bfloat16 holds exactly; z: zero point of 4-bit codes
template <int KIND>
__device__ __forceinline__ float unit_get(const RawUnit<KIND>& r, int e, float z)
{
    if constexpr (KIND == kCacheBf16) return e & 1 ? bf16_hi(r.w[e / 2]) : bf16_lo(r.w[e / 2]);
    else if constexpr (KIND == kCacheI8) return (float)(int8_t)(r.w[e / 4] >> (8 * (e & 3)));
    else return (float)((r.w[0] >> (4 * e)) & 15u) - z;
}

template <int KIND, int DP, int QR, bool PAGE16>
__global__ __launch_bounds__(64 * kTileWaves) __attribute__((amdgpu_waves_per_eu(DP == 256 ? 1 : 2, DP == 256 ? 1 : 2)))
void attention_tile_kernel(const AttnArgs a)
{
    using S = TileShape<DP>;
    constexpr int kRows = 32 * QR * kTileWaves;
    constexpr int kWords = S::kTokens * DP / 8;          // of 16 bytes, in a stage of k or v
    __shared__ __align__(16) u32x4 sk[2][kWords], sv[2][kWords];
    __shared__ __align__(16) float sks[2][S::kTokens], svs[2][S::kTokens];      // k's scale times scale2, v's scale
    __shared__ __align__(16) uint8_t sbad[2][2 * S::kSteps], sodd[2][2 * S::kSteps];          // by halves of 16 tokens, as v's units
    const CacheView& c = a.c;
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, half = lane >> 5;
    // blocks of one sequence and head follow each other at a distance of all of
    // them, so that they share an XCD's cache where their number is a multiple
    // of 8; a sequence's last rows, which see the most, come first
    uint32_t id = blockIdx.x;
    const uint32_t pairs = (uint32_t)c.heads * (uint32_t)a.s.seqs;
    const int h = (id % pairs) % (uint32_t)c.heads, b = (id % pairs) / (uint32_t)c.heads;
    id /= pairs;
    const int split = id % (uint32_t)a.splits;
    id /= (uint32_t)a.splits;
    const RowSpan r = seq_span(a.s, b);
    const int rows = r.n * a.group;                      // below 2^31 with all heads
    if (a.few_rows && rows <= a.few_rows) return;        // the other kernel's
    const uint8_t* kb = c.k + cache_bytes<KIND>(h * c.ld_head);
    const uint8_t* vb = c.v + cache_bytes<KIND>(h * c.ld_head);

    // what this thread stages: a unit of 8 tokens of k (first half of the threads) or of v
    const bool is_v = tid >= 128;
    const int su = tid % S::kUnits, so = (tid & 127u) / S::kUnits;               // unit, octet of tokens
    auto staged_token = [&](int e) { return is_v ? 16 * (so >> 1) + 4 * (so & 1) + (e & 3) + 8 * (e >> 2) : 8 * so + e; };
    const uint8_t* from = is_v ? vb : kb;
    const uint32_t* scales = is_v ? c.vs : c.ks;
    const bool unit_in = 8 * su < c.width;

    const int64_t row_tiles = (rows + kRows - 1) / kRows;
    for (int64_t at_tile = id; at_tile < row_tiles; at_tile += a.tiles) {
        const int64_t rt = row_tiles - 1 - at_tile;
        // this lane's rows, and of the wave's, whose positions grow
        int hi[QR], lo[QR];
        bf16x8 fq[QR][DP / 16];
#pragma unroll
        for (int x = 0; x < QR; ++x) {
            const int64_t rr = rt * kRows + (wave * QR + x) * 32 + col;
            const bool there = rr < rows;
            const int i = there ? (int)rr / a.group : 0;
            const int qh = h * a.group + (there ? (int)rr - i * a.group : 0);
            const int pos = r.pos(i);
            hi[x] = there ? (a.causal ? pos : r.len - 1) : -1;           // it sees lo .. hi
            lo[x] = a.window ? pos - a.window + 1 : 0;
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks)
                fq[x][ks] = __builtin_bit_cast(
                    bf16x8, ld_raw8<true, false>(a.q, (int64_t)(r.row0 + i) * a.ld_q + (int64_t)qh * c.width, 16 * ks + 8 * half,
                                                 c.width).v[0]);
        }
        int some_hi = -1, some_lo = INT32_MAX, all_hi = -1, all_lo = 0;   // some row sees some_lo .. some_hi, each all_lo .. all_hi
        const int64_t first_row = rt * kRows + wave * QR * 32;
        if (first_row < rows) {
            const int p0 = r.pos((int)first_row / a.group), p1 = r.pos(((int)min(first_row + 32 * QR, (int64_t)rows) - 1) / a.group);
            all_hi = a.causal ? p0 : r.len - 1;
            some_hi = a.causal ? p1 : r.len - 1;
            all_lo = a.window ? p1 - a.window + 1 : 0;
            some_lo = a.window ? p0 - a.window + 1 : 0;
        }
        int begin, end;
        const int i0 = (int)(rt * kRows) / a.group, i1 = ((int)min((int64_t)rows, (rt + 1) * kRows) - 1) / a.group;
        seen_span(a, r, i0, i1, begin, end);
        split_span(a.splits, split, begin, end);
        // tiles inside these bounds are seen whole by every row of the block
        const int block_hi = min(a.causal ? r.pos(i0) : r.len - 1, end - 1);
        const int block_lo = a.window ? r.pos(i1) - a.window + 1 : 0;

        RawUnit<KIND> raw[8];
        uint32_t word[8];
        uint32_t bad;
        auto load = [&](int p0) {
            bad = 0;
            int64_t page0 = 0;
            uint32_t slot0 = 0;
            if constexpr (PAGE16) {
                const uint32_t p = (uint32_t)min(p0 + (staged_token(0) & ~15), end - 1);
                const uint32_t entry = p / c.page_tokens;
                const int32_t page = cache_page(a.s, c, b, entry);
                if (page < 0) bad = 255u;
                page0 = page < 0 ? 0 : page;
                slot0 = (p - entry * c.page_tokens) & ~15u;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if constexpr (!PAGE16) {
                    const uint32_t p = (uint32_t)min(p0 + staged_token(e), end - 1);
                    const uint32_t entry = p / c.page_tokens;
                    const int32_t page = cache_page(a.s, c, b, entry);
                    if (page < 0) bad |= 1u << e;
                    page0 = page < 0 ? 0 : page;
                    slot0 = p - entry * c.page_tokens;
                }
                const uint32_t slot = PAGE16 ? slot0 + (staged_token(e) & 15) : slot0;
                const int64_t at = page0 * c.ld_page + (int64_t)slot * c.ld_token + 8 * su;
                raw[e] = RawUnit<KIND>{};
                if (unit_in) __builtin_memcpy(raw[e].w, __builtin_assume_aligned(from + cache_bytes<KIND>(at), sizeof(raw[e].w)), sizeof(raw[e].w));
                if constexpr (KIND != kCacheBf16) word[e] = scales[page0 * c.ld_sp + h * c.ld_sh + slot];
            }
        };
        auto stage = [&](int buf, int p0) {
            float z[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = KIND == kCacheI4 ? half_hi(word[e]) : 0.0f;
            if (su == 0) {
                if constexpr (KIND != kCacheBf16) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float s = KIND == kCacheI8 ? __builtin_bit_cast(float, word[e]) : half_lo(word[e]);
                        (is_v ? svs : sks)[buf][staged_token(e)] = is_v ? s : s * a.scale2;
                    }
                }
                if (is_v) sbad[buf][so] = (uint8_t)bad;
            }
            if (!is_v) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int t = 8 * so + e;
                    u32x4 o;
                    if constexpr (KIND == kCacheBf16) {
                        o = u32x4{raw[e].w[0], raw[e].w[1], raw[e].w[2], raw[e].w[3]};
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            o[i] = upper_pair(unit_get<KIND>(raw[e], 2 * i, z[e]), unit_get<KIND>(raw[e], 2 * i + 1, z[e]));
                    }
                    sk[buf][((t >> 5) * S::kUnits + su) * 32 + ((t & 31) ^ (su & 7))] = o;
                }
                return;
            }
            if constexpr (KIND == kCacheBf16) {
                uint32_t odd = 0;
                if (p0 < block_lo || p0 + S::kTokens - 1 > block_hi) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const uint32_t no = not_finite2(raw[e].w[w]);
                            raw[e].w[w] &= ~no;
                            odd |= no ? 1u << e : 0u;
                        }
                    odd = group_fold<S::kUnits>(odd, [](uint32_t p, uint32_t q) { return p | q; });
                }
                if (su == 0) sodd[buf][so] = (uint8_t)odd;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                u32x4 o;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (KIND == kCacheBf16)
                        o[i] = __builtin_amdgcn_perm(raw[2 * i + 1].w[e / 2], raw[2 * i].w[e / 2], e & 1 ? 0x07060302u : 0x05040100u);
                    else
                        o[i] = upper_pair(unit_get<KIND>(raw[2 * i], e, z[2 * i]), unit_get<KIND>(raw[2 * i + 1], e, z[2 * i + 1]));
                }
                const int part = e / S::kEach, dr = (e % S::kEach) * S::kUnits + su;
                sv[buf][(((so >> 1) * S::kParts + part) * 2 + (so & 1)) * 32 + dr] = o;
            }
        };

        f32x16 o[QR][S::kParts];
        float m[QR], l[QR];
#pragma unroll
        for (int x = 0; x < QR; ++x) {
            m[x] = neg_inf();
            l[x] = 0.0f;
#pragma unroll
            for (int p = 0; p < S::kParts; ++p)
#pragma unroll
                for (int v = 0; v < 16; ++v) o[x][p][v] = 0.0f;
        }
        auto first = [&](int buf, int sub, f32x16 (&acc)[QR]) {
#pragma unroll
            for (int x = 0; x < QR; ++x)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[x][v] = 0.0f;
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks) {
                const int u = 2 * ks + half;
                const bf16x8 fk = __builtin_bit_cast(bf16x8, sk[buf][(sub * S::kUnits + u) * 32 + (col ^ (u & 7))]);
#pragma unroll
                for (int x = 0; x < QR; ++x) acc[x] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fk, fq[x][ks], acc[x], 0, 0, 0);
            }
        };
        auto second = [&](int buf, int sub, int p0, bool whole, bool bad_tile, f32x16 (&acc)[QR]) {
            bf16x8 fp[QR][2];
#pragma unroll
            for (int x = 0; x < QR; ++x) {
                float y[16];
                uint32_t seen = 0xFFFFu, odd = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f32x4 ks = f32x4{a.scale2, a.scale2, a.scale2, a.scale2};
                    if constexpr (KIND != kCacheBf16) ks = *(const f32x4*)&sks[buf][32 * sub + 8 * j + 4 * half];
#pragma unroll
                    for (int k = 0; k < 4; ++k) y[4 * j + k] = acc[x][4 * j + k] * ks[k];
                }
                if (!whole || bad_tile) {
                    const uint32_t no = sbad[buf][4 * sub + half] | (uint32_t)sbad[buf][4 * sub + 2 + half] << 8;
                    if constexpr (KIND == kCacheBf16) odd = sodd[buf][4 * sub + half] | (uint32_t)sodd[buf][4 * sub + 2 + half] << 8;
#pragma unroll
                    for (int v = 0; v < 16; ++v) {
                        const int p = p0 + 32 * sub + 8 * (v >> 2) + 4 * half + (v & 3);
                        if ((no >> v) & 1u) y[v] = nan_f32();
                        if (!(p >= lo[x] && p <= hi[x] && p < end)) {
                            y[v] = neg_inf();
                            seen &= ~(1u << v);
                        }
                    }
                }
                float top = y[0];
#pragma unroll
                for (int v = 1; v < 16; ++v) top = fmaxf(top, y[v]);
                if (__any(top > m[x] + kRaise)) {
                    top = fmaxf(top, __shfl_xor(top, 32));
                    const float up = top > m[x] + kRaise ? top : m[x];
                    const float fac = up == m[x] ? 1.0f : exp2_fast(m[x] - up);
                    m[x] = up;
                    l[x] *= fac;
#pragma unroll
                    for (int p = 0; p < S::kParts; ++p) o[x][p] *= fac;
                }
                const float base = m[x] == neg_inf() ? 0.0f : m[x];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f32x4 vs;
                    if constexpr (KIND != kCacheBf16) vs = *(const f32x4*)&svs[buf][32 * sub + 8 * j + 4 * half];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int v = 4 * j + k;
                        float p = exp2_fast(y[v] - base);
                        l[x] += p;
                        if constexpr (KIND != kCacheBf16) p *= vs[k];
                        if (!whole || bad_tile) {
                            const bool sees = (seen >> v) & 1u;
                            if (KIND == kCacheBf16 && ((odd >> v) & 1u)) p = nan_f32();
                            if (!sees) p = 0.0f;
                        }
                        fp[x][v >> 3][v & 7] = (__bf16)p;
                    }
                }
            }
#pragma unroll
            for (int st = 0; st < 2; ++st)
#pragma unroll
                for (int p = 0; p < S::kParts; ++p) {
                    const bf16x8 fv = __builtin_bit_cast(bf16x8, sv[buf][(((2 * sub + st) * S::kParts + p) * 2 + half) * 32 + col]);
#pragma unroll
                    for (int x = 0; x < QR; ++x) o[x][p] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fv, fp[x][st], o[x][p], 0, 0, 0);
                }
        };

        if (begin < end) {
            load(begin);
            stage(0, begin);
        }
        __syncthreads();
        int buf = 0;
        for (int p0 = begin; p0 < end; p0 += S::kTokens, buf ^= 1) {
            const bool more = p0 + S::kTokens < end;
            if (more) load(p0 + S::kTokens);
            if (p0 <= some_hi && p0 + S::kTokens > some_lo) {
                const bool whole = all_lo <= p0 && p0 + S::kTokens - 1 <= all_hi && p0 + S::kTokens <= end;
                bool bad_tile = false;
#pragma unroll
                for (int i = 0; i < 2 * S::kSteps; i += 4) bad_tile |= *(const uint32_t*)&sbad[buf][i] != 0;
                f32x16 acc[2][QR];
                first(buf, 0, acc[0]);
#pragma unroll
                for (int sub = 0; sub < S::kSubs; ++sub) {
                    if (sub + 1 < S::kSubs) first(buf, sub + 1, acc[(sub + 1) & 1]);
                    second(buf, sub, p0, whole, bad_tile, acc[sub & 1]);
                }
            }
            if (more) stage(buf ^ 1, p0 + S::kTokens);
            __syncthreads();
        }

        // a lane holds, of its rows, units of 8 elements
#pragma unroll
        for (int x = 0; x < QR; ++x) {
            l[x] += __shfl_xor(l[x], 32);
            const int64_t rr = rt * kRows + (wave * QR + x) * 32 + col;
            if (rr >= rows) continue;
            const int64_t i = (int)rr / a.group, t = r.row0 + i;
            const int64_t qh = h * a.group + (rr - i * a.group), at = t * c.heads * a.group + qh;
            if (hi[x] >= a.s.capacity) l[x] = nan_f32();     // it sees tokens that the table does not hold
            const float inv = a.splits > 1 ? 1.0f : (l[x] == 0.0f ? 0.0f : 1.0f / l[x]);
            constexpr int kSlots = 16 / S::kEach;
#pragma unroll
            for (int k = 0; k < kSlots; ++k) {
                const int d = 8 * (8 * (k >> 2) + 4 * half + (k & 3));
                if (d >= c.width) continue;
                float e[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) e[j] = o[x][j / S::kEach][k + kSlots * (j % S::kEach)] * inv;
                if (a.splits > 1) {
                    float* po = a.part_o + (at * a.splits + split) * c.width + d;
                    *(f32x4*)po = f32x4{e[0], e[1], e[2], e[3]};
                    *(f32x4*)(po + 4) = f32x4{e[4], e[5], e[6], e[7]};
                } else {
                    st_row8<true, false>(a.out, t * a.ld_out + qh * c.width, d, c.width, e);
                }
            }
            if (half == 0) {
                if (a.splits > 1) *(f32x2*)(a.part_ml + 2 * (at * a.splits + split)) = f32x2{m[x], l[x]};
                else if (a.lse) a.lse[at] = row_lse(m[x], l[x]);
            }
        }
    }
}

// Joins the parts of every row, in the order of the parts: a wave to a row, 4
// elements of it to a lane.
__global__ __launch_bounds__(kBlock) void attention_join_kernel(const AttnArgs a, int64_t rows)
{
    const CacheView& c = a.c;
    const int lane = threadIdx.x & 63;
    const int heads = c.heads * a.group;
    for (int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); at < rows; at += (int64_t)gridDim.x * 4) {
        const int64_t t = at / heads;
        if (seq_of_row(a.s, t) < 0) continue;
        const float* ml = a.part_ml + 2 * at * a.splits;
        float m = neg_inf();
        for (int s = 0; s < a.splits; ++s) m = fmaxf(m, ml[2 * s]);
        float l = 0.0f;
        f32x4 o = {0, 0, 0, 0};
        for (int s = 0; s < a.splits; ++s) {
            const float ms = ml[2 * s], ls = ml[2 * s + 1];
            if (ls == 0.0f) continue;
            const float f = ms == neg_inf() ? ls : exp2_fast(ms - m);          // m of -inf: l is NaN
            l = __builtin_fmaf(ls, f, l);
            if (4 * lane < c.width) {
                const f32x4 v = *(const f32x4*)(a.part_o + (at * a.splits + s) * c.width + 4 * lane);
#pragma unroll
                for (int k = 0; k < 4; ++k) o[k] = __builtin_fmaf(v[k], f, o[k]);
            }
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        if (4 * lane < c.width) {
            const bf16x2 w[2] = {bf16x2{(__bf16)(o[0] * inv), (__bf16)(o[1] * inv)},
                                 bf16x2{(__bf16)(o[2] * inv), (__bf16)(o[3] * inv)}};
            __builtin_memcpy(a.out + t * a.ld_out + (at - t * heads) * c.width + 4 * lane, w, 8);
        }
        if (lane == 0 && a.lse) a.lse[at] = row_lse(m, l);
    }
}

}  // namespace echo
