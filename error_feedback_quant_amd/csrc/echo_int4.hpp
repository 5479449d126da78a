// echo_int4.hpp — gfx950 kernels of the linear layer with 4-bit weights: the
// quantizer of a row's groups, and the product for few tokens.
//
// Product: y[m][n] = sum_g s[n][g] (sum_{k in g} x[m][k] q[n][k]
//                                   - z[n][g] sum_{k in g} x[m][k]) + bias[n].
// A code becomes the bfloat16 16 + q with two instructions for two of them
// (shift and and-or: q goes to bits 3 .. 6 of the significand of 16.0), exact,
// and the matrix cores sum x (16 + q) and, with a row of ones in place of the
// weight, x itself; (16 + z) times the latter is taken off in fp32.  16 is the
// least offset that a bfloat16 holds beside four bits: the sums cancel by a
// factor of at most 31 / 15, where 128 + q would lose three bits more (fp32
// tokens, whose results are not rounded to bfloat16 afterwards, cancel most of
// it in the matrix cores already, see Int4Sums).
#pragma once

#include <type_traits>

#include "echo_kernels.hpp"
#include "echo_rows.hpp"

namespace echo {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Reductions over L lanes (4, 8, 16 or 32, aligned): inside a 16-lane row by
// DPP (the mirrors join halves whose lanes agree already), across two rows by
// a swizzle.  All lanes of the group have to be active.
template <int L, typename F>
__device__ __forceinline__ uint32_t group_fold(uint32_t v, F f)
{
    v = f(v, (uint32_t)dpp_i<0xB1>((int)v));                 // quad_perm 1,0,3,2
    v = f(v, (uint32_t)dpp_i<0x4E>((int)v));                 // quad_perm 2,3,0,1
    if constexpr (L >= 8) v = f(v, (uint32_t)dpp_i<0x141>((int)v));    // row_half_mirror
    if constexpr (L >= 16) v = f(v, (uint32_t)dpp_i<0x140>((int)v));   // row_mirror
    if constexpr (L >= 32) v = f(v, (uint32_t)__builtin_amdgcn_ds_swizzle((int)v, 0x401F));   // lane ^ 16
    return v;
}
template <int L>
__device__ __forceinline__ uint32_t group_max_u32(uint32_t v)
{
    return group_fold<L>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}

// 4-bit codes of a lane's 8 elements and the parameter word of its group of L
// lanes (the zero-aware quantizer; elements past the end are zeros, which its
// range holds anyway).  top: the lane's largest |u| as bits.
template <int L>
__device__ __forceinline__ uint32_t quantize4(const float (&u)[8], uint32_t top, uint32_t& word)
{
    float lo, hi;
    lane_stats<kZeroAware>(u, lo, hi);
    // the patterns of zeros and negative floats order as unsigned integers by
    // magnitude, those of zeros and positive floats as integers
    const uint32_t l = group_max_u32<L>(__builtin_bit_cast(uint32_t, lo));
    const uint32_t h = group_fold<L>(__builtin_bit_cast(uint32_t, hi),
                                     [](uint32_t a, uint32_t b) { return (uint32_t)max((int)a, (int)b); });
    const QParams p = make_params<4, kZeroAware>(__builtin_bit_cast(float, l), __builtin_bit_cast(float, h));
    const bool bad = group_max_u32<L>(top) >= 0x7F800000u;
    word = bad ? 0x7E00u : p.word;                           // NaN, zero point 0
    uint32_t q = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) q |= (uint32_t)quant1<4, kZeroAware>(u[e], p) << (4 * e);
    return bad ? 0u : q;
}

struct QuantGroupArgs {
    const void* x;
    uint8_t* q;
    uint32_t* p;
    int64_t ldx, ldq, ldp, T;
    int K;
    int shift;              // 1 << shift threads share a row (at least a group's, at most a block)
};

// A thread takes 8 elements, the L lanes of a group find its range together.
// One pass over memory.
template <int L, bool BF16>
__global__ __launch_bounds__(kBlock) void quantize_groups_kernel(const QuantGroupArgs a)
{
    const int per = 1 << a.shift, rows = kBlock >> a.shift;
    const int c0 = threadIdx.x & (per - 1), g = threadIdx.x & (L - 1);
    const int chunks = (int)(((int64_t)a.K + 8 * L - 1) / (8 * L)) * L;      // whole groups
    for (int64_t t0 = (int64_t)blockIdx.x * rows; t0 < a.T; t0 += (int64_t)gridDim.x * rows) {
        const int64_t t = t0 + (threadIdx.x >> a.shift);
        const bool in = t < a.T;
        for (int c = c0 + per * (int)blockIdx.y; c < chunks; c += per * (int)gridDim.y) {
            const int k = 8 * c;
            const Raw8<BF16> raw = ld_raw8<BF16, true>(a.x, in ? t * a.ldx : 0, k, in ? a.K : 0);
            float u[8];
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                u[e] = raw_get(raw, e);
                top = max(top, abs_bits(u[e]));
            }
            uint32_t word;
            uint32_t q = quantize4<L>(u, top, word);
            if (!in || k >= a.K) continue;
            uint8_t* to = a.q + t * a.ldq + 4 * (int64_t)c;
            if (k + 8 <= a.K) {
                __builtin_memcpy(to, &q, 4);
            } else {
                const int n = a.K - k;                       // 1 .. 7
                q &= (1u << (4 * n)) - 1u;
                for (int i = 0; i < (n + 1) / 2; ++i) to[i] = (uint8_t)(q >> (8 * i));
            }
            if (g == 0) a.p[t * a.ldp + c / L] = word;
        }
    }
}

// ------------------------------------------------------------- few tokens --
//
// A block of 8 waves takes 16 channels and 16 MT tokens; its waves take
// every eighth unit of K (128 elements, or a group of 256) and their sums meet
// in LDS in a fixed order.  x is the first operand, so a lane keeps one
// channel, whose scales and zero points it needs, and four tokens of a tile.
//
// The weight passes once, without LDS: a lane loads 16 bytes, 32 codes of its
// channel, and the four lanes of a channel exchange words so that each has the
// codes that stand beside its 8 elements of x in an MFMA.  So both loads are
// whole: 64 contiguous bytes of a row for four lanes (with
// the codes as loaded and x in their order, 16-byte pieces at distances of 64,
// 27 x 1001 x 3583 took 11.4 us, so 10.0).  A block's loads of DEPTH units are
// on their way together, codes, parameters and tokens.

constexpr int kInt4Waves = 8;
constexpr int kInt4Threads = 64 * kInt4Waves;

struct Int4Args {
    const void* x;
    const uint8_t* w;
    const uint32_t* p;
    const float* bias;
    void* y;
    int64_t M, N, ldx, ldw, ldp, ldy;
    int K;
    int bf16;               // of y
};

// codes 2i and 2i + 8 .. : the pairs (0, 4), (1, 5), (2, 6), (3, 7) of a word's
// nibbles as bfloat16 16 + q
// (bias: two 16.0 in a register; an and-or takes only one literal)
__device__ __forceinline__ bf16x8 codes_bf16(uint32_t w, uint32_t bias)
{
    u32x4 r;
    r.x = ((w << 3) & 0x00780078u) | bias;
    r.y = ((w >> 1) & 0x00780078u) | bias;
    r.z = ((w >> 5) & 0x00780078u) | bias;
    r.w = ((w >> 9) & 0x00780078u) | bias;
    return __builtin_bit_cast(bf16x8, r);
}

// two floats' upper halves as a pair
__device__ __forceinline__ uint32_t upper_pair(float lo, float hi)
{
    return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, hi), __builtin_bit_cast(uint32_t, lo), 0x07060302u);
}

// x's 8 elements in the order of codes_bf16, as P bfloat16 parts that sum to
// them: one for bf16, three (8 + 8 + 8 bits) for fp32.  Truncation makes each
// part, so each rest is exact.
template <bool BF16, int P>
__device__ __forceinline__ void x_parts(const Raw8<BF16>& r, bf16x8 (&f)[P])
{
    if constexpr (BF16) {
        u32x4 o;
        o.x = __builtin_amdgcn_perm(r.v[0].z, r.v[0].x, 0x05040100u);
        o.y = __builtin_amdgcn_perm(r.v[0].z, r.v[0].x, 0x07060302u);
        o.z = __builtin_amdgcn_perm(r.v[0].w, r.v[0].y, 0x05040100u);
        o.w = __builtin_amdgcn_perm(r.v[0].w, r.v[0].y, 0x07060302u);
        f[0] = __builtin_bit_cast(bf16x8, o);
    } else {
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = raw_get(r, i);
            v[2 * i + 1] = raw_get(r, i + 4);
        }
#pragma unroll
        for (int p = 0; p < P; ++p) {
            u32x4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o[i] = upper_pair(v[2 * i], v[2 * i + 1]);
                v[2 * i] -= __builtin_bit_cast(float, o[i] << 16);
                v[2 * i + 1] -= __builtin_bit_cast(float, o[i] & 0xFFFF0000u);
            }
            f[p] = __builtin_bit_cast(bf16x8, o);
        }
    }
}

// 16 bytes of codes from byte `at` of a row of `bytes`, zeros past its end
__device__ __forceinline__ u32x4 ld_codes16(const uint8_t* row, int64_t at, int64_t bytes)
{
    u32x4 v = {0, 0, 0, 0};
    if (at + 16 <= bytes) {
        __builtin_memcpy(&v, row + at, 16);
    } else {
        for (int i = 0; i < 16 && at + i < bytes; ++i) v[i / 4] |= (uint32_t)row[at + i] << (8 * (i & 3));
    }
    return v;
}

// Word f of the 16 lanes g (g, f from 0 to 3) goes to word g of the lanes f.
__device__ __forceinline__ void turn4(u32x4& w)
{
    const auto a = __builtin_amdgcn_permlane32_swap(w.x, w.z, false, false);     // upper half of the first with the lower of the second
    const auto b = __builtin_amdgcn_permlane32_swap(w.y, w.w, false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);   // odd rows of the first with even ones of the second
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    w = u32x4{c[0], c[1], d[0], d[1]};
}

// A lane's four sums of x times codes (or ones).  fp32 x comes in three parts,
// of which the first has nearly all of the sum: the others have sums of their
// own, so that it is rounded once for a fragment and not three times.  The
// middle of the codes' range, 16 + 8, is taken off after every fragment as well,
// by a product with -24: what is left for the zero points to cancel is a few
// units in the place of 24.  Over drawn shapes with fp32 x the error, relative to
// y's norm, was up to 1.5e-6 without either and is up to 2.5e-7 so.
// At K = 4096, groups of 128: neither 1.3e-6 (us for 1 x 4096 x 4096, 64 x 8192
// x 8192: 7.5, 52), sums apart 3.5e-7 (8.2, 54), both 1.2e-7 (8.8, 56), which is
// what a product in fp32 is off by.
template <int PARTS>
struct Int4Sums {
    f32x4 high = {0, 0, 0, 0}, low = {0, 0, 0, 0};
    __device__ __forceinline__ void add(const bf16x8 (&x)[PARTS], const bf16x8& w)
    {
        high = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[0], w, high, 0, 0, 0);
#pragma unroll
        for (int p = 1; p < PARTS; ++p) low = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[p], w, low, 0, 0, 0);
    }
    __device__ __forceinline__ float get(int v) const { return PARTS > 1 ? high[v] + low[v] : high[v]; }
};
__device__ __forceinline__ bf16x8 eight_of(float v)          // a bfloat16 value, eight times
{
    const uint32_t w = __builtin_bit_cast(uint32_t, v) >> 16;
    return __builtin_bit_cast(bf16x8, u32x4{w * 0x10001u, w * 0x10001u, w * 0x10001u, w * 0x10001u});
}

template <int GROUP, int MT, int DEPTH, bool BF16>
__global__ __launch_bounds__(kInt4Threads) void linear_int4_kernel(const Int4Args a)
{
    constexpr int kPart = BF16 ? 1 : 3;
    constexpr int kUnit = GROUP < 128 ? 128 : GROUP;
    constexpr int kLoads = kUnit / 128, kGroups = kUnit / GROUP;        // of a unit
    constexpr int kFrags = kUnit / 32;
    __shared__ f32x4 part[kInt4Waves][MT][64];
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t col = lane & 15u, g = lane >> 4;
    const int64_t n0 = 16 * (int64_t)blockIdx.x, m0 = (int64_t)blockIdx.y * (16 * MT);
    const int64_t bytes = ((int64_t)a.K + 1) / 2;
    // channels and tokens past the last one repeat it: their sums are not stored
    const int64_t channel = min(n0 + col, a.N - 1);
    const uint8_t* wr = a.w + channel * a.ldw;
    const uint32_t* pr = a.p + channel * a.ldp;
    int64_t xr[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) xr[t] = min(m0 + 16 * t + col, a.M - 1) * a.ldx;
    uint32_t bias = 0x41804180u, one = 0x3F803F80u;          // two 16.0, two 1.0
    asm("" : "+v"(bias), "+v"(one));
    const u32x4 one4 = {one, one, one, one};
    const bf16x8 ones = __builtin_bit_cast(bf16x8, one4), centre = eight_of(-24.0f);

    struct Unit {
        u32x4 w[kLoads];
        uint32_t p[kGroups];
        Raw8<BF16> x[MT][kFrags];
    };
    auto k_of = [&](int u, int f) __attribute__((always_inline)) {     // first element of the lane's fragment f
        return u * kUnit + 32 * f + 8 * (int)g;
    };
    auto code_of = [&](int u, int s) __attribute__((always_inline)) {  // first byte of its load s of codes
        return (int64_t)(u * kUnit + 128 * s + 32 * (int)g) / 2;
    };
    f32x4 y[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) y[t] = f32x4{0, 0, 0, 0};
    auto take = [&](Unit& d) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < kLoads; ++s) turn4(d.w[s]);
#pragma unroll
        for (int q = 0; q < kGroups; ++q) {
            Int4Sums<kPart> acc[MT], xs[MT];
#pragma unroll
            for (int f = q * (kFrags / kGroups); f < (q + 1) * (kFrags / kGroups); ++f) {
                const bf16x8 fw = codes_bf16(d.w[f / 4][f % 4], bias);
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    bf16x8 fx[kPart];
                    x_parts<BF16, kPart>(d.x[t][f], fx);
                    xs[t].add(fx, ones);
                    acc[t].add(fx, fw);
                    if constexpr (kPart > 1) acc[t].add(fx, centre);
                }
            }
            const uint32_t word = d.p[q];
            const float z = (kPart > 1 ? 8.0f : -16.0f) - half_hi(word);
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    y[t][v] = __builtin_fmaf(half_lo(word), __builtin_fmaf(z, xs[t].get(v), acc[t].get(v)), y[t][v]);
        }
    };

    const int full = a.K / kUnit;                            // units inside K
    auto load = [&](Unit& d, int u) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < kLoads; ++s) __builtin_memcpy(&d.w[s], wr + code_of(u, s), 16);
        __builtin_memcpy(d.p, pr + (int64_t)u * kGroups, 4 * kGroups);
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int f = 0; f < kFrags; ++f)
                __builtin_memcpy(d.x[t][f].v, (const char*)a.x + (xr[t] + k_of(u, f)) * (BF16 ? 2 : 4), sizeof(d.x[t][f].v));
    };
    const int mine = full > (int)wave ? (full - (int)wave + kInt4Waves - 1) / kInt4Waves : 0;     // units of this wave
    auto unit_of = [&](int i) { return (int)wave + kInt4Waves * i; };
    for (int i0 = 0; i0 < mine; i0 += DEPTH) {
        Unit d[DEPTH];
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) load(d[i], unit_of(min(i0 + i, mine - 1)));           // without a condition they go out together
#pragma unroll
        for (int i = 0; i < DEPTH; ++i)
            if (i == 0 || i0 + i < mine) take(d[i]);
    }
    if (full * kUnit < a.K && (uint32_t)full % kInt4Waves == wave) {   // the unit that K ends in: x is 0 past K
        Unit d;
#pragma unroll
        for (int s = 0; s < kLoads; ++s) d.w[s] = ld_codes16(wr, code_of(full, s), bytes);
#pragma unroll
        for (int q = 0; q < kGroups; ++q) d.p[q] = full * kUnit + q * GROUP < a.K ? pr[(int64_t)full * kGroups + q] : 0u;
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int f = 0; f < kFrags; ++f) d.x[t][f] = ld_raw8<BF16, true>(a.x, xr[t], k_of(full, f), a.K);
        take(d);
    }
    // lane l holds channel l % 16 and tokens 4 (l / 16) .. + 3 of each tile
#pragma unroll
    for (int t = 0; t < MT; ++t) part[wave][t][lane] = y[t];
    __syncthreads();
    for (uint32_t i = tid; i < 64 * MT; i += kInt4Threads) {
        const uint32_t tile = i >> 6, l = i & 63u;
        f32x4 s = part[0][tile][l];
#pragma unroll
        for (int w = 1; w < kInt4Waves; ++w) s += part[w][tile][l];
        const int64_t m = m0 + 16 * tile + 4 * (l >> 4);
        const int64_t n = n0 + (l & 15u);
        if (n >= a.N) continue;
        const float b = a.bias ? a.bias[n] : 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (m + e < a.M) st_elem(a.y, a.bf16, (m + e) * a.ldy + n, a.bias ? s[e] + b : s[e]);
    }
}

// ------------------------------------------------------------- more tokens --
//
// Every block of channels reads all of x, and a fragment of x is 64 bytes of 16
// rows, which lie in one channel of the cache where a row is a multiple of 4 KB:
// 14 bytes a clock and CU (64 x 8192 x 8192: 41.5 us of a product whose matrix
// instructions take 6).  So more tokens are laid out once as the
// fragments that the blocks read, with the sums of its groups beside them:
// whole kilobytes, no permutations and a third fewer matrix instructions
// (23.5 us and 4.5 for the arrangement).

struct Int4Tiles {
    Int4Args a;
    bf16x8* x;              // [units][tiles][fragments][parts][64 lanes]
    f32x4* xs;              // [units][groups][tiles][4]: sums of tokens 4 g .. + 3
    int units, tiles;       // tiles of 16 tokens, a multiple of MT
};

template <int GROUP, bool BF16>
__global__ __launch_bounds__(kBlock) void arrange_int4_kernel(const Int4Tiles b)
{
    constexpr int kPart = BF16 ? 1 : 3, kUnit = GROUP < 128 ? 128 : GROUP, kGroups = kUnit / GROUP, kFrags = kUnit / 32;
    const uint32_t lane = threadIdx.x & 63u, col = lane & 15u, g = lane >> 4;
    const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (id >= (int64_t)b.units * b.tiles) return;
    const int u = (int)(id / b.tiles), t = (int)(id % b.tiles);
    const int64_t m = 16 * (int64_t)t + col;
    const bool in = m < b.a.M;
    Int4Sums<kPart> xs[kGroups];
#pragma unroll
    for (int f = 0; f < kFrags; ++f) {
        bf16x8 fx[kPart];
        x_parts<BF16, kPart>(ld_raw8<BF16, true>(b.a.x, in ? m * b.a.ldx : 0, u * kUnit + 32 * f + 8 * (int)g, in ? b.a.K : 0), fx);
#pragma unroll
        for (int p = 0; p < kPart; ++p) b.x[((id * kFrags + f) * kPart + p) * 64 + lane] = fx[p];
        xs[f / (kFrags / kGroups)].add(fx, eight_of(1.0f));
    }
    if (col == 0) {
#pragma unroll
        for (int q = 0; q < kGroups; ++q) b.xs[(((int64_t)u * kGroups + q) * b.tiles + t) * 4 + g] = f32x4{xs[q].get(0), xs[q].get(1), xs[q].get(2), xs[q].get(3)};
    }
}

template <int GROUP, int MT, int NT, int P>
__global__ __launch_bounds__(kInt4Threads) __attribute__((amdgpu_waves_per_eu(2))) void linear_int4_tile_kernel(const Int4Tiles b)
{
    constexpr int kUnit = GROUP < 128 ? 128 : GROUP, kLoads = kUnit / 128, kGroups = kUnit / GROUP, kFrags = kUnit / 32;
    __shared__ f32x4 part[kInt4Waves][MT * NT][64];
    const Int4Args& a = b.a;
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t col = lane & 15u, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * NT);
    const int t0 = (int)blockIdx.y * MT;
    const int64_t bytes = ((int64_t)a.K + 1) / 2;
    const uint8_t* wr[NT];
    const uint32_t* pr[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int64_t n = min(n0 + 16 * j + col, a.N - 1);
        wr[j] = a.w + n * a.ldw;
        pr[j] = a.p + n * a.ldp;
    }
    uint32_t bias = 0x41804180u;
    asm("" : "+v"(bias));
    const bf16x8 centre = eight_of(-24.0f);
    f32x4 y[MT][NT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < NT; ++j) y[t][j] = f32x4{0, 0, 0, 0};
    auto unit = [&](int u, u32x4 (&w)[NT][kLoads], const uint32_t (&word)[NT][kGroups]) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int s = 0; s < kLoads; ++s) turn4(w[j][s]);
#pragma unroll
        for (int q = 0; q < kGroups; ++q) {
            Int4Sums<P> acc[MT][NT];
            f32x4 xs[MT];
#pragma unroll
            for (int t = 0; t < MT; ++t) xs[t] = b.xs[(((int64_t)u * kGroups + q) * b.tiles + t0 + t) * 4 + g];
#pragma unroll
            for (int f = q * (kFrags / kGroups); f < (q + 1) * (kFrags / kGroups); ++f) {
                bf16x8 fw[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) fw[j] = codes_bf16(w[j][f / 4][f % 4], bias);
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    bf16x8 fx[P];
#pragma unroll
                    for (int p = 0; p < P; ++p) fx[p] = b.x[((((int64_t)u * b.tiles + t0 + t) * kFrags + f) * P + p) * 64 + lane];
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        acc[t][j].add(fx, fw[j]);
                        if constexpr (P > 1) acc[t][j].add(fx, centre);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const float z = (P > 1 ? 8.0f : -16.0f) - half_hi(word[j][q]);
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        y[t][j][v] = __builtin_fmaf(half_lo(word[j][q]), __builtin_fmaf(z, xs[t][v], acc[t][j].get(v)), y[t][j][v]);
            }
        }
    };
    auto byte_of = [&](int u, int s) { return (int64_t)(u * kUnit + 128 * s + 32 * (int)g) / 2; };
    const int full = a.K / kUnit;                            // units whose codes are all there
    for (int u = wave; u < full; u += kInt4Waves) {
        u32x4 w[NT][kLoads];
        uint32_t word[NT][kGroups];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int s = 0; s < kLoads; ++s) __builtin_memcpy(&w[j][s], wr[j] + byte_of(u, s), 16);
            __builtin_memcpy(word[j], pr[j] + (int64_t)u * kGroups, 4 * kGroups);
        }
        unit(u, w, word);
    }
    if (full < b.units && (uint32_t)full % kInt4Waves == wave) {
        u32x4 w[NT][kLoads];
        uint32_t word[NT][kGroups];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int s = 0; s < kLoads; ++s) w[j][s] = ld_codes16(wr[j], byte_of(full, s), bytes);
#pragma unroll
            for (int q = 0; q < kGroups; ++q) word[j][q] = full * kUnit + q * GROUP < a.K ? pr[j][(int64_t)full * kGroups + q] : 0u;
        }
        unit(full, w, word);
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int j = 0; j < NT; ++j) part[wave][t * NT + j][lane] = y[t][j];
    __syncthreads();
    for (uint32_t i = tid; i < 64 * MT * NT; i += kInt4Threads) {
        const uint32_t tile = i >> 6, l = i & 63u;
        f32x4 s = part[0][tile][l];
#pragma unroll
        for (int w = 1; w < kInt4Waves; ++w) s += part[w][tile][l];
        const int64_t m = 16 * (int64_t)(t0 + tile / NT) + 4 * (l >> 4), n = n0 + 16 * (tile % NT) + (l & 15u);
        if (n >= a.N) continue;
        const float c = a.bias ? a.bias[n] : 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (m + e < a.M) st_elem(a.y, a.bf16, (m + e) * a.ldy + n, a.bias ? s[e] + c : s[e]);
    }
}

}  // namespace echo
