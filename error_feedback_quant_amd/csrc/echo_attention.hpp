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
// takes p_j t_j times d_j.  8-bit codes are exact in bfloat16.  Of 4-bit codes,
//  - the kernel for few rows, where a code is used a few times only, takes
//    16 + c (echo_int4.hpp): two instructions for two codes.  The offset is taken
//    off the score through the sum of q, and off the output through
//    sum_j p_j t_j (16 + w_j), one number a row, in fp32;
//  - the kernel for many rows takes c - z, made once in fp32 when a tile is
//    staged: no offset, and small integers are exact in bfloat16.
// p_j t_j is rounded to bfloat16 (half a unit of 2^-8), the type of the matrix
// operand, where there are many rows; few rows have what that leaves as a second
// operand.  m, l and all sums are fp32.
//
// Both products take tokens as the rows (of k) or the depth (of v) of the
// first operand and query rows as the columns of the second, so a lane keeps
// one query row throughout: its scores, weights, m and l stay in its own
// registers from the first product to the second, where they are the second
// operand as they are.
//
// A masked token has weight 0, but 0 times an infinity or a NaN in v is NaN.
// Codes are finite, and a scale enters through p_j t_j, which a mask sets to 0;
// so does a zero point: in few rows with the scale, in many, where it is part of
// the operand, one that is no number is staged as the scale NaN.  In a bfloat16
// cache the elements of v that are no numbers are set to 0 where a tile is
// masked in part, and the rows that see their token get the weight NaN.
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
    int few_rows;           // rows up to which a sequence is the few-row kernel's, 0: the launched kernel takes all
    uint32_t tiles;         // row tiles: of a sequence (few rows), of the call (many)
    // parts of a row's tokens and where they leave their sums, for either kernel
    struct Parts {
        int splits;
        float* o;           // [rows][splits][width]
        float* ml;          // [rows][splits][2]
    } few, tile;
};

// A row's number among those that leave parts.  Where both kernels run, the
// few-row one has few_rows for each sequence and head of the cache.
__device__ __forceinline__ int64_t few_part(const AttnArgs& a, int64_t at, int b, int h, int64_t row)
{
    return a.few_rows ? ((int64_t)b * a.c.heads + h) * a.few_rows + row : at;
}

typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRaise = 8.0f;   // a row's m follows its largest score when that is 2^8 above it

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float nan_f32() { return __builtin_bit_cast(float, 0x7FC00000u); }
__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// largest / sum over the lanes that share a query row: lane % 16 with ROWS = 4, lane % 32 with 2
__device__ __forceinline__ float row_max16(float v)      // within 16 lanes
{
    v = fmaxf(v, __builtin_bit_cast(float, dpp_i<0xB1>(__builtin_bit_cast(int, v))));
    v = fmaxf(v, __builtin_bit_cast(float, dpp_i<0x4E>(__builtin_bit_cast(int, v))));
    v = fmaxf(v, __builtin_bit_cast(float, dpp_i<0x141>(__builtin_bit_cast(int, v))));
    return fmaxf(v, __builtin_bit_cast(float, dpp_i<0x140>(__builtin_bit_cast(int, v))));
}
template <int ROWS>
__device__ __forceinline__ float rows_max(float v)
{
    if constexpr (ROWS == 4) v = fmaxf(v, __shfl_xor(v, 16));
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
    // one sequence to a block: said to the compiler, which sees loads
    RowSpan r;
    const int e = __builtin_amdgcn_readfirstlane(s.starts[b + 1]);
    r.row0 = __builtin_amdgcn_readfirstlane(s.starts[b]);
    r.len = __builtin_amdgcn_readfirstlane(max(s.lens[b], 0));
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

// A row's reference m and its sum l.  Scores come as z = y - m straight from
// one fma; m follows the largest score when that is 2^8 above it, which leaves
// most tiles without a rescaling, and weights of up to 2^8 are as exact as any.
// Rows are raised one by one, so that no row's rounding goes by another's.
struct RowSum {
    float minus_m = 0.0f;   // 0 before the first score
    float over = -__builtin_inff();     // raise m where z passes this: kRaise, before the first score -infinity
    float l = 0.0f;
    __device__ __forceinline__ float m() const { return over < 0.0f ? neg_inf() : -minus_m; }
};

// Makes room for scores z (N of a lane's row, the largest top): afterwards
// none is over kRaise.  scale(f) multiplies what was summed before.
template <int ROWS, int N, typename F>
__device__ __forceinline__ void row_raise(RowSum& r, float (&z)[N], float top, F scale)
{
    if (__any(top > r.over)) {
        top = rows_max<ROWS>(top);
        const bool up = top > r.over;
        const float by = up ? top : 0.0f;
        const float f = up ? (r.over < 0.0f ? 0.0f : exp2_fast(-by)) : 1.0f;
        r.minus_m -= by;
        r.over = up ? kRaise : r.over;
        r.l *= f;
#pragma unroll
        for (int v = 0; v < N; ++v) z[v] -= by;
        scale(f);
    }
}

// 8 floats as bfloat16, two to an instruction
__device__ __forceinline__ bf16x8 to_bf16x8(const float* p)
{
    bf16x2 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf16x2{(__bf16)p[2 * i], (__bf16)p[2 * i + 1]};
    bf16x8 r;
    __builtin_memcpy(&r, w, 16);
    return r;
}

// lse of a row whose sums are whole
__device__ __forceinline__ float row_lse(float m, float l) { return (m + __builtin_log2f(l)) * kLn2; }

// l of a row whose sums are whole and that sees tokens up to `last`.  The
// largest score has the weight 1 when m rises to it, so l is 0 only where no
// score was above -infinity; a row that sees tokens all the same is NaN, as
// exp(-infinity - -infinity) is.
__device__ __forceinline__ float whole_sum(float l, int last) { return l == 0.0f && last >= 0 ? nan_f32() : l; }

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
    uint32_t ks, vs;            // of token lane % 8 among the 8 of the lane's row
};

// f(0) .. f(7) with the number as a constant
template <typename F>
__device__ __forceinline__ void unroll8(F f)
{
    using std::integral_constant;
    f(integral_constant<int, 0>{}); f(integral_constant<int, 1>{}); f(integral_constant<int, 2>{}); f(integral_constant<int, 3>{});
    f(integral_constant<int, 4>{}); f(integral_constant<int, 5>{}); f(integral_constant<int, 6>{}); f(integral_constant<int, 7>{});
}

// v of lane E of the octet's lanes (8, or the 16 of a row, of which every
// eighth holds the same): a broadcast within the row
template <int UNITS, int E>
__device__ __forceinline__ uint32_t octet_lane(uint32_t v)
{
    const uint32_t a = (uint32_t)dpp_i<0x150 + E>((int)v);   // row_newbcast
    if constexpr (UNITS >= 16) return a;
    const uint32_t b = (uint32_t)dpp_i<0x158 + E>((int)v);
    return threadIdx.x & 8u ? b : a;
}

// 8 elements of k (words) as bfloat16
template <int KIND>
__device__ __forceinline__ bf16x8 k_frag(const uint32_t* w, uint32_t bias)
{
    u32x4 o;
    if constexpr (KIND == kCacheBf16) {
        o = u32x4{w[0], w[1], w[2], w[3]};
    } else if constexpr (KIND == kCacheI8) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = upper_pair((float)(int8_t)(w[i / 2] >> (16 * (i & 1))), (float)(int8_t)(w[i / 2] >> (16 * (i & 1) + 8)));
    } else {
        return codes_bf16(w[0], bias);
    }
    return __builtin_bit_cast(bf16x8, o);
}

// element f of 8 tokens' pieces of v
template <int KIND, int WORDS>
__device__ __forceinline__ bf16x8 v_frag(const uint32_t (*v)[WORDS], int f, uint32_t bias)
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
            o[i] = ((at ? h >> (at - 3) : h << 3) & 0x00780078u) | bias;
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

// waves on a SIMD that a tile's and the sums' registers leave room for
constexpr int few_waves(int dp) { return dp == 64 ? 4 : (dp == 128 ? 3 : 2); }

// PAGE16: pages are a multiple of 16 tokens, so the 16 tokens of a tile's half
// lie in one page; otherwise every lane looks its tokens up.
template <int KIND, int DP, bool PAGE16>
__global__ __launch_bounds__(64 * kFewAttnWaves) __attribute__((amdgpu_waves_per_eu(few_waves(DP))))
void attention_few_kernel(const AttnArgs a)
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
    // the row tiles of a part are 8 blocks apart: they share an XCD's cache
    uint32_t id = blockIdx.x / 8 / a.tiles * 8 + blockIdx.x % 8;
    const int split = id % (uint32_t)a.few.splits;
    id /= (uint32_t)a.few.splits;
    const int h = id % (uint32_t)c.heads;
    const int b = id / (uint32_t)c.heads;
    if (b >= a.s.seqs) return;
    const RowSpan r = seq_span(a.s, b);
    const int rows = r.n * a.group;                      // below 2^31 with all heads
    if (a.few_rows && rows > a.few_rows) return;         // the other kernel's
    const uint8_t* kb = c.k + cache_bytes<KIND>(h * c.ld_head);
    const uint8_t* vb = c.v + cache_bytes<KIND>(h * c.ld_head);
    const int64_t token_bytes = cache_bytes<KIND>(c.ld_token);
    const uint32_t koff = (uint32_t)(col * token_bytes + cache_bytes<KIND>(S::kE * g));      // for PAGE16, whose host check
    const uint32_t voff = (uint32_t)(4 * g * token_bytes + cache_bytes<KIND>(S::kVE * col)); // keeps them in 32 bits

    for (int64_t rt = blockIdx.x / 8 % a.tiles; rt * kFewRows < rows; rt += a.tiles) {
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
        split_span(a.few.splits, split, begin, end);

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

        // Page numbers come a tile before the loads that need them.
        struct Pages {
            int32_t n[PAGE16 ? 2 : 10];
        };
        auto entry_of = [&](int p) { return (uint32_t)min(p, end - 1) / c.page_tokens; };
        auto lookup = [&](int p0) __attribute__((always_inline)) {
            Pages pg;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if constexpr (PAGE16) {
                    pg.n[u] = cache_page(a.s, c, b, entry_of(p0 + 16 * u));
                } else {
                    pg.n[8 + u] = cache_page(a.s, c, b, entry_of(p0 + 16 * u + col));
#pragma unroll
                    for (int e = 0; e < 4; ++e) pg.n[4 * u + e] = cache_page(a.s, c, b, entry_of(p0 + 16 * u + 4 * g + e));
                }
            }
            return pg;
        };
        // one token's k (load j) and v; at: 8 elements, or what is left of the width
        auto take_k = [&](uint32_t (&w)[S::kKWords], const uint8_t* at, int j) __attribute__((always_inline)) {
            const int d = S::kE * (4 * j + g);
            if (d + S::kE <= c.width) {
                __builtin_memcpy(w, __builtin_assume_aligned(at, 4), 4 * S::kKWords);
            } else {                                         // q is 0 past the width, and so has k to be
                constexpr int kWords8 = S::kKWords * 8 / S::kE;             // of 8 elements
#pragma unroll
                for (int i = 0; i < S::kKWords; ++i) w[i] = d + i / kWords8 * 8 < c.width ? ((const uint32_t*)at)[i] : 0u;
            }
        };
        auto take_v = [&](uint32_t (&w)[S::kVWords], const uint8_t* at, int p) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < S::kVWords; ++i) w[i] = 0;
            if (128 * p + S::kVE * col < c.width) __builtin_memcpy(w, at, S::kVBytes);
        };
        constexpr int kLoadBytes = 4 * 4 * S::kKWords;       // of k, from one load of a lane to its next
        constexpr int kPieceBytes = 16 * S::kVBytes;
        auto load = [&](FewTile<KIND, DP>& f, int p0, const Pages& pg) __attribute__((always_inline)) {
            uint32_t kbad = 0, bad = 0;                      // tokens without a place, by bits: their scores are NaN
            int64_t mine = 0;                                // entry of token lane % 8's scales
            if constexpr (PAGE16) {
                // a base for 16 tokens in scalar registers, and the lane's offsets
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int32_t page = __builtin_amdgcn_readfirstlane(pg.n[u]);
                    if (page < 0) bad |= 15u << (4 * u), kbad |= 1u << u;
                    const int64_t at = page < 0 ? 0 : page;
                    const uint32_t slot = (uint32_t)min(p0 + 16 * u, end - 1) % c.page_tokens & ~15u;
                    const int64_t row = cache_bytes<KIND>(at * c.ld_page + slot * c.ld_token);
                    const uint8_t *kr = kb + row, *vr = vb + row;
#pragma unroll
                    for (int j = 0; j < S::kLoads; ++j) take_k(f.k[u][j], kr + j * kLoadBytes + koff, j);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int p = 0; p < S::kPieces; ++p) take_v(f.v[4 * u + e][p], vr + e * token_bytes + p * kPieceBytes + voff, p);
                    if constexpr (KIND != kCacheBf16) {
                        const int64_t sr = at * c.ld_sp + h * c.ld_sh + slot;
                        mine = u == 0 || (lane & 4u) ? sr : mine;
                    }
                }
                mine += 4 * g + (lane & 3u);
            } else {
                auto place = [&](int t, int32_t page, int64_t& o, int64_t& s) __attribute__((always_inline)) {
                    const uint32_t slot = (uint32_t)min(t, end - 1) % c.page_tokens;
                    const int64_t at = page < 0 ? 0 : page;
                    o = at * c.ld_page + (int64_t)slot * c.ld_token;
                    s = at * c.ld_sp + h * c.ld_sh + slot;
                    return page < 0;
                };
                int64_t o, s;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (place(p0 + 16 * u + col, pg.n[8 + u], o, s)) kbad |= 1u << u;
#pragma unroll
                    for (int j = 0; j < S::kLoads; ++j) take_k(f.k[u][j], kb + cache_bytes<KIND>(o + S::kE * (4 * j + g)), j);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (place(p0 + 16 * (e / 4) + 4 * g + (e & 3), pg.n[e], o, s)) bad |= 1u << e;
#pragma unroll
                    for (int p = 0; p < S::kPieces; ++p) take_v(f.v[e][p], vb + cache_bytes<KIND>(o + 128 * p + S::kVE * col), p);
                    mine = (int)(lane & 7u) == e ? s : mine;
                }
            }
            if constexpr (KIND != kCacheBf16) {
                f.ks = c.ks[mine];
                f.vs = c.vs[mine];
            }
            if (__any((bad | kbad) != 0)) {
                if (KIND != kCacheBf16 && (bad >> (lane & 7u)) & 1u) f.ks = KIND == kCacheI8 ? 0x7FC00000u : 0x7E00u;
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    if (KIND == kCacheBf16 && (kbad >> u) & 1u) f.k[u][0][0] = 0x7FC07FC0u;
            }
        };

        f32x4 o[kFrags];
#pragma unroll
        for (int f = 0; f < kFrags; ++f) o[f] = f32x4{0, 0, 0, 0};
        int p0 = begin + kFewTile * (int)wave;
        RowSum sum;
        float off = 0.0f, off16 = 0.0f;                      // what zero points and 1/16 of the offset add to every element
        uint32_t bias = 0x41804180u;                         // two 16.0: in a register, an and-or takes one literal
        asm("" : "+v"(bias));

        auto take = [&](FewTile<KIND, DP>& f) __attribute__((always_inline)) {
            f32x4 acc[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                // the offset 16 of 4-bit codes is off from the start
                const float first = KIND == kCacheI4 ? -16.0f * qsum : 0.0f;
                acc[u] = f32x4{first, first, first, first};
#pragma unroll
                for (int st = 0; st < kSteps; ++st) {
                    constexpr int kPer = S::kE / 8, kW = S::kKWords / kPer;
                    acc[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k_frag<KIND>(&f.k[u][st / kPer][kW * (st % kPer)], bias),
                                                                     fq[st], acc[u], 0, 0, 0);
                }
            }
            float z[8];
            uint32_t ks[8], vs[8];
            if constexpr (KIND != kCacheBf16)
                unroll8([&](auto e) {
                    ks[e] = octet_lane<16, e>(f.ks);
                    vs[e] = octet_lane<16, e>(f.vs);
                });
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float s = acc[e / 4][e % 4];
                if constexpr (KIND == kCacheBf16) z[e] = __builtin_fmaf(s, a.scale2, sum.minus_m);
                else if constexpr (KIND == kCacheI8) z[e] = __builtin_fmaf(s * a.scale2, __builtin_bit_cast(float, ks[e]), sum.minus_m);
                else z[e] = __builtin_fmaf(__builtin_fmaf(half_hi(ks[e]), -qsum, s) * a.scale2, half_lo(ks[e]), sum.minus_m);
            }
            // Tiles that are masked in part: the weight is 0 for a score of
            // -infinity, and so has what it is multiplied with to be a number.
            if (!(__all(!there || (lo <= p0 && p0 + kFewTile - 1 <= hi)) && p0 + kFewTile <= end)) {
                asm volatile("");                            // a branch, not selects in every tile
                uint32_t odd = 0;                            // tokens whose v holds no number
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
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int p = p0 + 16 * (e / 4) + 4 * g + (e & 3);
                    const bool sees = (p >= lo) & (p <= hi) & (p < end);
                    if (KIND == kCacheBf16 && ((odd >> e) & 1u)) z[e] = nan_f32();
                    z[e] = sees ? z[e] : neg_inf();
                    if constexpr (KIND != kCacheBf16) vs[e] = sees ? vs[e] : 0u;     // of this row and token
                }
            }
            float top = z[0];
#pragma unroll
            for (int e = 1; e < 8; ++e) top = fmaxf(top, z[e]);
            row_raise<4>(sum, z, top, [&](float by) {
                off *= by;
                off16 *= by;
#pragma unroll
                for (int j = 0; j < kFrags; ++j) o[j] *= by;
            });
            float p[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                p[e] = exp2_fast(z[e]);
                sum.l += p[e];
                if constexpr (KIND == kCacheI8) p[e] *= __builtin_bit_cast(float, vs[e]);
                if constexpr (KIND == kCacheI4) p[e] = __builtin_fmaf(p[e], half_lo(vs[e]), 0.0f);
            }
            if constexpr (KIND == kCacheI4) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    off = __builtin_fmaf(p[e], half_hi(vs[e]), off);
                    off16 += p[e];
                }
            }
            // The weights in two parts of 8 bits each: the output then carries no
            // rounding but its own.  In one part its error was up to 1.5 times
            // that; the second costs little where the loads are what is waited for
            // (64 sequences over up to 16384 tokens: 185 us in the place of 172).
            const bf16x8 fp = to_bf16x8(p);
            const u32x4 high = __builtin_bit_cast(u32x4, fp);
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] -= e & 1 ? bf16_hi(high[e / 2]) : bf16_lo(high[e / 2]);
            const bf16x8 fl = to_bf16x8(p);
#pragma unroll
            for (int pc = 0; pc < S::kPieces; ++pc) {
                uint32_t v[8][S::kVWords];
#pragma unroll
                for (int e = 0; e < 8; ++e)
#pragma unroll
                    for (int w = 0; w < S::kVWords; ++w) v[e][w] = f.v[e][pc][w];
#pragma unroll
                for (int j = 0; j < S::kVE; ++j) {
                    const bf16x8 fv = v_frag<KIND, S::kVWords>(v, j, bias);
                    f32x4& sums = o[S::kVE * pc + j];
                    sums = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fv, fp, sums, 0, 0, 0);
                    sums = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fv, fl, sums, 0, 0, 0);
                }
            }
        };
        // Other waves cover a wave's wait for its tile: three on a SIMD that load
        // and multiply in turn (64 tokens over up to 16384 in 4 bits, the weights
        // in one part: 172 us, 3.9 TB/s; two or three waves with their next tile
        // on its way 178 and 209).
        constexpr int kStep = kFewTile * kFewAttnWaves;
        if (p0 < end) {
            Pages pg = lookup(p0);
            for (; p0 < end; p0 += kStep) {
                FewTile<KIND, DP> f;
                load(f, p0, pg);
                pg = lookup(p0 + kStep);
                take(f);
            }
        }

        // the waves' sums to the largest m
        const float m = sum.m(), l = rows4_sum(sum.l);
        if constexpr (KIND == kCacheI4) off = rows4_sum(__builtin_fmaf(16.0f, off16, off));
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
            if (a.few.splits > 1) {
                const int64_t part = few_part(a, at, b, h, row) * a.few.splits + split;
                float* po = a.few.o + part * c.width + d;
                *(f32x4*)po = f32x4{e[0], e[1], e[2], e[3]};
                *(f32x4*)(po + 4) = f32x4{e[4], e[5], e[6], e[7]};
                if (d == 0) *(f32x2*)(a.few.ml + 2 * part) = f32x2{mm, ll};
            } else {
                ll = whole_sum(ll, last);
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
// A block of W waves takes 32 W rows of one sequence and head of the cache,
// 32 to a wave, and walks over the tokens in tiles of 2048 W / DP.  A
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

template <int DP, int W>
struct TileShape {
    static constexpr int kTokens = 2048 * W / DP;        // of a tile
    static constexpr int kUnits = DP / 8;                // of 8 elements
    static constexpr int kSubs = kTokens / 32;           // 32 tokens: the rows of a first product
    static constexpr int kSteps = kTokens / 16;          // 16 tokens: the depth of a second one
    static constexpr int kParts = DP / 32;               // 32 elements: the rows of a second one
    static constexpr int kEach = 32 / kUnits;            // elements of a unit in a part
};

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

template <int KIND, int DP, int W, bool PAGE16>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(DP == 256 ? 1 : 2, DP == 256 ? 1 : 2)))
void attention_tile_kernel(const AttnArgs a)
{
    using S = TileShape<DP, W>;
    constexpr int kRows = 32 * W;
    constexpr int kWords = S::kTokens * DP / 8;          // of 16 bytes, in a stage of k or v
    __shared__ __align__(16) u32x4 sk[2][kWords], sv[2][kWords];
    __shared__ __align__(16) float sks[2][S::kTokens], svs[2][S::kTokens];      // k's scale times scale2, v's scale
    __shared__ uint8_t sodd[2][2 * S::kSteps];           // tokens whose v holds no number, by v's octets
    const CacheView& c = a.c;
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, half = lane >> 5;
    // Heads are the fastest number: where they are a multiple of 8, all blocks
    // of a head share an XCD's cache.  Row tiles have numbers by their first
    // row in the whole call plus one for each sequence, so that the launch
    // needs no count of them and those that are there follow each other (with
    // blocks that have nothing to do between them, a chunk of 512 tokens beside
    // 7 single ones took 390 us, in this order 170 then); a sequence's last rows,
    // which see the most, come first.
    uint32_t id = blockIdx.x;
    const int h = id % (uint32_t)c.heads;
    id /= (uint32_t)c.heads;
    const int64_t v = id % a.tiles;
    const int split = id / a.tiles;
    auto tile_base = [&](int b) { return (int64_t)a.s.starts[b] * a.group / kRows + b; };
    const int b = last_at_most(a.s.seqs, v, tile_base);
    const RowSpan r = seq_span(a.s, b);
    const int rows = r.n * a.group;                      // below 2^31 with all heads
    if (a.few_rows && rows <= a.few_rows) return;        // the other kernel's
    const uint8_t* kb = c.k + cache_bytes<KIND>(h * c.ld_head);
    const uint8_t* vb = c.v + cache_bytes<KIND>(h * c.ld_head);

    // what this thread stages: a unit of 8 tokens, of k in the first half of
    // the waves and of v in the others
    const bool is_v = wave >= W / 2;
    const int su = tid % S::kUnits, so = (tid & (32 * W - 1)) / S::kUnits;       // unit, octet of tokens
    const int token0 = is_v ? 16 * (so >> 1) + 4 * (so & 1) : 8 * so;            // of the octet, then
    auto token_step = [&](int e) { return is_v ? (e & 3) + 8 * (e >> 2) : e; };
    const uint8_t* from = (is_v ? vb : kb) + cache_bytes<KIND>(8 * su);
    const uint32_t* scales = (is_v ? c.vs : c.ks) + h * c.ld_sh;
    const bool unit_in = 8 * su < c.width;
    const int64_t token_bytes = cache_bytes<KIND>(c.ld_token);
    // where k's unit of the octet's first token goes, in bytes; token e then lies at an exclusive or with 16 e
    const uint32_t k_at = 16u * (((token0 >> 5) * S::kUnits + su) * 32 + (token0 & 31) + (su & 7));

    const int64_t rt = ((int64_t)rows + kRows - 1) / kRows - 1 - (v - ((int64_t)r.row0 * a.group / kRows + b));
    if (rt < 0 || rt * kRows >= rows) return;
    {
        // this lane's row
        const int64_t rr = rt * kRows + wave * 32 + col;
        const bool there = rr < rows;
        const int i = there ? (int)rr / a.group : 0;
        const int64_t t = r.row0 + i;
        const int qh = h * a.group + (there ? (int)rr - i * a.group : 0);
        const int pos = r.pos(i);
        const int hi = there ? (a.causal ? pos : r.len - 1) : -1;            // it sees lo .. hi
        const int lo = a.window ? pos - a.window + 1 : 0;
        bf16x8 fq[DP / 16];
#pragma unroll
        for (int ks = 0; ks < DP / 16; ++ks)
            fq[ks] = __builtin_bit_cast(
                bf16x8, ld_raw8<true, false>(a.q, t * a.ld_q + (int64_t)qh * c.width, 16 * ks + 8 * half, c.width).v[0]);
        int some_hi = -1, some_lo = INT32_MAX;               // no row sees further than this
        const int64_t first_row = rt * kRows + wave * 32;
        if (first_row < rows) {
            some_hi = a.causal ? r.pos(((int)min(first_row + 32, (int64_t)rows) - 1) / a.group) : r.len - 1;
            some_lo = a.window ? r.pos((int)first_row / a.group) - a.window + 1 : 0;
        }
        int begin, end;
        const int i0 = (int)(rt * kRows) / a.group, i1 = ((int)min((int64_t)rows, (rt + 1) * kRows) - 1) / a.group;
        seen_span(a, r, i0, i1, begin, end);
        split_span(a.tile.splits, split, begin, end);
        // tiles inside these bounds are seen whole by every row of the block
        const int block_hi = min(a.causal ? r.pos(i0) : r.len - 1, end - 1);
        const int block_lo = a.window ? r.pos(i1) - a.window + 1 : 0;
        auto whole = [&](int p0) { return block_lo <= p0 && p0 + S::kTokens - 1 <= block_hi; };

        RawUnit<KIND> raw[8];
        uint32_t word = 0;                                   // scale or parameters of the octet's token su % 8
        uint32_t bad;                                        // tokens without a place, by bits: their scores are NaN
        auto load = [&](int p0) __attribute__((always_inline)) {
            auto lookup = [&](int t, int64_t& page, uint32_t& slot) __attribute__((always_inline)) {
                const uint32_t p = (uint32_t)min(p0 + t, end - 1);
                const uint32_t entry = p / c.page_tokens;
                page = cache_page(a.s, c, b, entry);
                slot = p - entry * c.page_tokens;
                const bool none = page < 0;
                page = none ? 0 : page;
                return none;
            };
            int64_t page;
            uint32_t slot;
            if constexpr (PAGE16) {
                bad = lookup(token0 & ~15, page, slot) ? 255u : 0u;
                slot = (slot & ~15u) + (token0 & 15);
                if constexpr (KIND != kCacheBf16) word = scales[page * c.ld_sp + slot + token_step(su & 7)];
                const uint8_t* at = from + cache_bytes<KIND>(page * c.ld_page + slot * c.ld_token);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    raw[e] = RawUnit<KIND>{};
                    if (unit_in) __builtin_memcpy(raw[e].w, __builtin_assume_aligned(at, sizeof(raw[e].w)), sizeof(raw[e].w));
                    at += token_bytes * (e == 3 && is_v ? 5 : 1);
                }
            } else {
                bad = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (lookup(token0 + token_step(e), page, slot)) bad |= 1u << e;
                    raw[e] = RawUnit<KIND>{};
                    const uint8_t* at = from + cache_bytes<KIND>(page * c.ld_page + slot * c.ld_token);
                    if (unit_in) __builtin_memcpy(raw[e].w, __builtin_assume_aligned(at, sizeof(raw[e].w)), sizeof(raw[e].w));
                }
                if constexpr (KIND != kCacheBf16) {
                    lookup(token0 + token_step(su & 7), page, slot);
                    word = scales[page * c.ld_sp + slot];
                }
            }
        };
        auto stage = [&](int buf, int p0) __attribute__((always_inline)) {
            float z[8];                                      // zero points
            if constexpr (KIND == kCacheI4) {
                // One that is no number would make the operand none, which a
                // weight of 0 does not undo: its token's scale is NaN instead,
                // and a mask takes that off (slots behind the last token and
                // tokens before the window are staged as they lie there).
                if ((word & 0x7C000000u) == 0x7C000000u) word = 0x7E00u;
                unroll8([&](auto e) { z[e] = half_hi(octet_lane<S::kUnits, e>(word)); });
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) z[e] = 0.0f;
            }
            if constexpr (KIND != kCacheBf16) {
                if (su < 8) {
                    float s = KIND == kCacheI8 ? __builtin_bit_cast(float, word) : half_lo(word);
                    if ((bad >> su) & 1u) s = nan_f32();
                    (is_v ? svs : sks)[buf][token0 + token_step(su)] = is_v ? s : s * a.scale2;
                }
            }
            if (!is_v) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    u32x4 o;
                    if constexpr (KIND == kCacheBf16) {
                        o = u32x4{raw[e].w[0], raw[e].w[1], raw[e].w[2], raw[e].w[3]};
                        if ((bad >> e) & 1u) o = u32x4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            o[i] = upper_pair(unit_get<KIND>(raw[e], 2 * i, z[e]), unit_get<KIND>(raw[e], 2 * i + 1, z[e]));
                    }
                    *(u32x4*)((uint8_t*)sk[buf] + (k_at ^ (16u * e))) = o;
                }
                return;
            }
            if constexpr (KIND == kCacheBf16) {
                uint32_t odd = 0;
                if (!whole(p0)) {
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

        f32x16 o[S::kParts];
#pragma unroll
        for (int p = 0; p < S::kParts; ++p)
#pragma unroll
            for (int v = 0; v < 16; ++v) o[p][v] = 0.0f;
        RowSum sum;
        // scores of 32 tokens before they are scaled
        auto first = [&](int buf, int sub) __attribute__((always_inline)) {
            f32x16 acc;
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[v] = 0.0f;
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks) {
                const int u = 2 * ks + half;
                const bf16x8 fk = __builtin_bit_cast(bf16x8, sk[buf][(sub * S::kUnits + u) * 32 + (col ^ (u & 7))]);
                acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fk, fq[ks], acc, 0, 0, 0);
            }
            return acc;
        };
        // z of them, with the mask, and the largest
        auto scores = [&](auto masked, int buf, int sub, int p0, const f32x16& acc, float (&z)[16], uint32_t& seen)
            __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f32x4 ks = f32x4{a.scale2, a.scale2, a.scale2, a.scale2};
                if constexpr (KIND != kCacheBf16) ks = *(const f32x4*)&sks[buf][32 * sub + 8 * j + 4 * half];
#pragma unroll
                for (int k = 0; k < 4; ++k) z[4 * j + k] = __builtin_fmaf(acc[4 * j + k], ks[k], sum.minus_m);
            }
            if constexpr (decltype(masked)::value) {
                seen = 0;
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    const int p = p0 + 32 * sub + 8 * (v >> 2) + 4 * half + (v & 3);
                    const bool sees = (p >= lo) & (p <= hi) & (p < end);
                    z[v] = sees ? z[v] : neg_inf();
                    seen |= sees ? 1u << v : 0u;
                }
            }
            float top = z[0];
#pragma unroll
            for (int v = 1; v < 16; ++v) top = fmaxf(top, z[v]);
            return top;
        };
        // the weights as the second product's operands
        auto weights = [&](auto masked, int buf, int sub, const float (&z)[16], uint32_t seen, bf16x8 (&fp)[2])
            __attribute__((always_inline)) {
            uint32_t odd = 0;                                // tokens whose v holds no number
            if constexpr (decltype(masked)::value && KIND == kCacheBf16)
                odd = sodd[buf][4 * sub + half] | (uint32_t)sodd[buf][4 * sub + 2 + half] << 8;
            float p[16];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f32x4 vs;
                if constexpr (KIND != kCacheBf16) vs = *(const f32x4*)&svs[buf][32 * sub + 8 * j + 4 * half];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int v = 4 * j + k;
                    p[v] = exp2_fast(z[v]);
                    sum.l += p[v];
                    if constexpr (KIND != kCacheBf16) p[v] *= vs[k];
                    if constexpr (decltype(masked)::value) {
                        if (KIND == kCacheBf16 && ((odd >> v) & 1u)) p[v] = nan_f32();
                        if (!((seen >> v) & 1u)) p[v] = 0.0f;
                    }
                }
            }
            // One part of 8 bits: the error is up to 1.4 times that of an output
            // rounded once (0.0024 of the norm against 0.0017, 8192 over 8192 in 8
            // bits).  A second part, as few rows have it, doubles the second product
            // and the conversions: 614 us become 819, and 512 tokens beside 7
            // sequences 148 become 164.
            fp[0] = to_bf16x8(p);
            fp[1] = to_bf16x8(p + 8);
        };
        auto second = [&](int buf, int sub, const bf16x8 (&fp)[2]) __attribute__((always_inline)) {
#pragma unroll
            for (int st = 0; st < 2; ++st)
#pragma unroll
                for (int p = 0; p < S::kParts; ++p) {
                    const bf16x8 fv = __builtin_bit_cast(bf16x8, sv[buf][(((2 * sub + st) * S::kParts + p) * 2 + half) * 32 + col]);
                    o[p] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fv, fp[st], o[p], 0, 0, 0);
                }
        };
        // The matrix cores work while the weights of one 32 tokens are made,
        // on the scores of the next, and then on the weights while those
        // scores are scaled and compared; the order is asked for, since
        // matrix instructions in a row would hold up the wave's others.
        auto products = [&](auto masked, int buf, int p0) __attribute__((always_inline)) {
            float z[16];
            uint32_t seen = 0xFFFFu;
            f32x16 acc = first(buf, 0);
            float top = scores(masked, buf, 0, p0, acc, z, seen);
#pragma unroll
            for (int sub = 0; sub < S::kSubs; ++sub) {
                row_raise<2>(sum, z, top, [&](float by) __attribute__((always_inline)) {
#pragma unroll
                    for (int p = 0; p < S::kParts; ++p) o[p] *= by;
                });
                bf16x8 fp[2];
                if (sub + 1 < S::kSubs) acc = first(buf, sub + 1);
                weights(masked, buf, sub, z, seen, fp);
                second(buf, sub, fp);
                if (sub + 1 < S::kSubs) {
                    top = scores(masked, buf, sub + 1, p0, acc, z, seen);
                    if constexpr (!decltype(masked)::value) {
                        __builtin_amdgcn_sched_group_barrier(0x100, 10, 0);                // reads of LDS go ahead
#pragma unroll
                        for (int i = 0; i < DP / 16; ++i) {
                            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);             // a matrix product
                            __builtin_amdgcn_sched_group_barrier(0x402, 56 * 16 / DP, 0);  // what the vector unit does meanwhile
                            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                        }
#pragma unroll
                        for (int i = 0; i < 2 * S::kParts; ++i) {
                            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                            __builtin_amdgcn_sched_group_barrier(0x402, 12 / S::kParts, 0);
                            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                        }
                    }
                }
            }
        };

        if (begin < end) {
            load(begin);
            stage(0, begin);
        }
        __syncthreads();
        // masked tiles stand at both ends of the part
        int buf = 0, p0 = begin;
        auto turn = [&](auto masked) __attribute__((always_inline)) {
            const bool more = p0 + S::kTokens < end;
            if (more) load(p0 + S::kTokens);
            if (!decltype(masked)::value || (p0 <= some_hi && p0 + S::kTokens > some_lo)) products(masked, buf, p0);
            if (more) stage(buf ^ 1, p0 + S::kTokens);
            __syncthreads();
            p0 += S::kTokens;
            buf ^= 1;
        };
        while (p0 < end) {
            while (p0 < end && !whole(p0)) turn(std::true_type{});
            while (p0 < end && whole(p0)) turn(std::false_type{});
        }

        // a lane holds, of its row, units of 8 elements
        float l = sum.l + __shfl_xor(sum.l, 32);
        if (there) {
            const int64_t at = t * c.heads * a.group + qh;
            if (hi >= a.s.capacity) l = nan_f32();           // it sees tokens that the table does not hold
            const bool parts = a.tile.splits > 1;
            if (!parts) l = whole_sum(l, hi);
            const float inv = parts ? 1.0f : (l == 0.0f ? 0.0f : 1.0f / l);
            constexpr int kSlots = 16 / S::kEach;
#pragma unroll
            for (int k = 0; k < kSlots; ++k) {
                const int d = 8 * (8 * (k >> 2) + 4 * half + (k & 3));
                if (d >= c.width) continue;
                float e[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) e[j] = o[j / S::kEach][k + kSlots * (j % S::kEach)] * inv;
                if (parts) {
                    float* po = a.tile.o + (at * a.tile.splits + split) * c.width + d;
                    *(f32x4*)po = f32x4{e[0], e[1], e[2], e[3]};
                    *(f32x4*)(po + 4) = f32x4{e[4], e[5], e[6], e[7]};
                } else {
                    st_row8<true, false>(a.out, t * a.ld_out + (int64_t)qh * c.width, d, c.width, e);
                }
            }
            if (half == 0) {
                if (parts) *(f32x2*)(a.tile.ml + 2 * (at * a.tile.splits + split)) = f32x2{sum.m(), l};
                else if (a.lse) a.lse[at] = row_lse(sum.m(), l);
            }
        }
    }
}

// Joins the parts of every row, in a fixed order: a wave to a row, whose lanes
// first take a part each for the common m and the parts' factors; then half a
// wave takes every other part, with kAhead loads on their way.  4 or 8 elements
// to a lane.
template <int DP>
__global__ __launch_bounds__(kBlock) void attention_join_kernel(const AttnArgs a, int64_t rows)
{
    constexpr int kE = DP <= 128 ? 4 : 8, kAhead = 4;
    const CacheView& c = a.c;
    const int lane = threadIdx.x & 63, half = lane >> 5, d = kE * (lane & 31);
    const int heads = c.heads * a.group;
    for (int64_t at = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); at < rows; at += (int64_t)gridDim.x * 4) {
        const int64_t t = at / heads;
        const int qh = (int)(at - t * heads);
        const int b = last_at_most(a.s.seqs, t, [&](int i) { return (int64_t)a.s.starts[i]; });
        if (!takes_row(a.s, b, t)) continue;
        const RowSpan r = seq_span(a.s, b);
        const int i = (int)(t - r.row0);
        const bool is_few = a.tile.splits == 0 || (a.few_rows && r.n * a.group <= a.few_rows);
        const AttnArgs::Parts& p = is_few ? a.few : a.tile;
        const int splits = p.splits;
        if (splits <= 1) continue;                           // written by its kernel
        const int h = qh / a.group;
        const int64_t part = (is_few ? few_part(a, at, b, h, (int64_t)i * a.group + (qh - h * a.group)) : at) * splits;
        const float* ml = p.ml + 2 * part;
        const float* po = p.o + part * c.width + d;
        // the parts' m, and their l at the common m; at most 64 parts
        float m = neg_inf(), l = 0.0f;
        if (lane < splits) {
            const f32x2 v = *(const f32x2*)(ml + 2 * lane);
            m = v.x;
            l = v.y;
        }
        const float top = rows_max<4>(row_max16(m));
        const float f = l == 0.0f ? 0.0f : (m == neg_inf() ? l : exp2_fast(m - top));     // m of -inf: l is NaN
        const float sum = whole_sum(wave_sum(l * f), a.causal ? r.pos(i) : r.len - 1);
        float o[kE] = {};
        const bool in = d < c.width;
        for (int s0 = 0; s0 < splits; s0 += 2 * kAhead) {
            f32x4 v[kAhead][kE / 4];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int s = min(s0 + 2 * i + half, splits - 1);
#pragma unroll
                for (int k = 0; k < kE / 4; ++k) v[i][k] = in ? *(const f32x4*)(po + (int64_t)s * c.width + 4 * k) : f32x4{0, 0, 0, 0};
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int s = s0 + 2 * i + half;
                const float fs = __shfl(f, min(s, splits - 1));
                if (s < splits && fs != 0.0f) {
#pragma unroll
                    for (int k = 0; k < kE; ++k) o[k] = __builtin_fmaf(v[i][k / 4][k % 4], fs, o[k]);
                }
            }
        }
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        uint32_t w[kE / 2];
#pragma unroll
        for (int k = 0; k < kE; k += 2) {
            const float x = (o[k] + __shfl_xor(o[k], 32)) * inv, y = (o[k + 1] + __shfl_xor(o[k + 1], 32)) * inv;
            w[k / 2] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)x, (__bf16)y});
        }
        if (half == 0 && in) __builtin_memcpy(a.out + t * a.ld_out + (int64_t)qh * c.width + d, w, sizeof(w));
        if (lane == 0 && a.lse) a.lse[at] = row_lse(top, sum);
    }
}

}  // namespace echo
