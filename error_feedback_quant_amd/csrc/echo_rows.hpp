// echo_rows.hpp — rows of a matrix held in registers: the loads, stores and
// reductions that the token quantizer and the block norms share.
//
// A row is taken by G threads (a wave, or a whole block) as chunks of 8
// consecutive elements, chunk j of thread g at element 8 (g + G j): 16 bytes
// of bf16 or 32 of fp32, so a wave's load is contiguous.  Rows start anywhere
// (gfx950 loads 16 bytes at any alignment of their elements).  TAIL is set
// where a row's length is no multiple of 8: the chunk that the row ends in is
// then read and written element by element.
#pragma once

#include "echo_kernels.hpp"

namespace echo {

__device__ __forceinline__ float ld_elem(const void* p, bool bf16, int64_t i)
{
    return bf16 ? __builtin_bit_cast(float, (uint32_t)((const uint16_t*)p)[i] << 16) : ((const float*)p)[i];
}
__device__ __forceinline__ void st_elem(void* p, bool bf16, int64_t i, float v)
{
    if (bf16) ((uint16_t*)p)[i] = __builtin_bit_cast(uint16_t, (__bf16)v);
    else ((float*)p)[i] = v;
}

// 8 elements as they lie in memory: 4 dwords of bf16 or 8 of fp32.  Kept raw
// until they are used, so that every load of a row is out before the first
// is waited for.
template <bool BF16>
struct Raw8 {
    u32x4 v[BF16 ? 1 : 2];
};

template <bool BF16, bool TAIL>
__device__ __forceinline__ Raw8<BF16> ld_raw8(const void* base, int64_t row, int k, int K)
{
    Raw8<BF16> r;
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) r.v[i] = u32x4{0, 0, 0, 0};
    if (k + 8 <= K) {
        __builtin_memcpy(r.v, (const char*)base + (row + k) * (BF16 ? 2 : 4), sizeof(r.v));
    } else if (TAIL && k < K) {
#pragma unroll
        for (int i = 0; i < 7; ++i) {
            if (k + i >= K) continue;
            if constexpr (BF16) r.v[0][i / 2] |= (uint32_t)((const uint16_t*)base)[row + k + i] << (16 * (i & 1));
            else r.v[i / 4][i % 4] = ((const uint32_t*)base)[row + k + i];
        }
    }
    return r;
}

template <bool BF16>
__device__ __forceinline__ float raw_get(const Raw8<BF16>& r, int e)
{
    if constexpr (BF16) {
        const uint32_t w = r.v[0][e / 2];
        return __builtin_bit_cast(float, (e & 1) ? (w & 0xFFFF0000u) : (w << 16));
    } else {
        return __builtin_bit_cast(float, (uint32_t)r.v[e / 4][e % 4]);
    }
}

template <bool BF16, bool TAIL>
__device__ __forceinline__ void st_row8(void* base, int64_t row, int k, int K, const float (&v)[8])
{
    if (k + 8 <= K) {
        if constexpr (BF16) {
            bf16x2 o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = bf16x2{(__bf16)v[2 * e], (__bf16)v[2 * e + 1]};
            __builtin_memcpy((uint16_t*)base + row + k, o, 16);
        } else {
            __builtin_memcpy((float*)base + row + k, v, 32);
        }
    } else if (TAIL && k < K) {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (k + i < K) st_elem(base, BF16, row + k + i, v[i]);
    }
}

// ---- a token's 8-bit scale and codes

constexpr float kI8Tiny = 0x1p-100f;         // smallest token magnitude that sets a scale

// max of |x| by bit pattern: the patterns of non-negative floats order as
// unsigned integers, with NaN above infinity above every finite value
__device__ __forceinline__ uint32_t abs_bits(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFFu; }

struct TokenScale {
    float scale, inv;
};
__device__ __forceinline__ TokenScale token_scale(uint32_t amax_bits)
{
    if (amax_bits >= 0x7F800000u) return {__builtin_bit_cast(float, 0x7FC00000u), 0.0f};
    const float a = fmaxf(__builtin_bit_cast(float, amax_bits), kI8Tiny);
    return {a / 127.0f, 127.0f / a};
}
// code of x under a token's inv; inv == 0 marks a token without one
__device__ __forceinline__ int token_code(float x, float inv)
{
    return inv == 0.0f ? 0 : (int)__builtin_rintf(x * inv);
}

// 8-bit codes
template <bool TAIL>
__device__ __forceinline__ void st_codes8(int8_t* base, int64_t row, int k, int K, const int (&q)[8])
{
    if (k + 8 <= K) {
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e / 4] |= (uint32_t)(q[e] & 255) << (8 * (e & 3));
        __builtin_memcpy(base + row + k, w, 8);
    } else if (TAIL && k < K) {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (k + i < K) base[row + k + i] = (int8_t)q[i];
    }
}

// Reductions over a wave: four steps inside each 16-lane row, then the rows'
// results by readlane, in a fixed order; every lane ends with the result.
__device__ __forceinline__ float wave_sum(float v)
{
    v += __builtin_bit_cast(float, dpp_i<0xB1>(__builtin_bit_cast(int, v)));    // quad_perm 1,0,3,2
    v += __builtin_bit_cast(float, dpp_i<0x4E>(__builtin_bit_cast(int, v)));    // quad_perm 2,3,0,1
    v += __builtin_bit_cast(float, dpp_i<0x124>(__builtin_bit_cast(int, v)));   // row_ror 4
    v += __builtin_bit_cast(float, dpp_i<0x128>(__builtin_bit_cast(int, v)));   // row_ror 8
    const int b = __builtin_bit_cast(int, v);
    const float r0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 0));
    const float r1 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 16));
    const float r2 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 32));
    const float r3 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 48));
    return (r0 + r1) + (r2 + r3);
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v)
{
    v = max(v, (uint32_t)dpp_i<0xB1>((int)v));
    v = max(v, (uint32_t)dpp_i<0x4E>((int)v));
    v = max(v, (uint32_t)dpp_i<0x124>((int)v));
    v = max(v, (uint32_t)dpp_i<0x128>((int)v));
    const uint32_t r0 = __builtin_amdgcn_readlane((int)v, 0), r1 = __builtin_amdgcn_readlane((int)v, 16);
    const uint32_t r2 = __builtin_amdgcn_readlane((int)v, 32), r3 = __builtin_amdgcn_readlane((int)v, 48);
    return max(max(r0, r1), max(r2, r3));
}

// The same over the G threads of a row.  A row of one wave needs no LDS; a
// row of a whole block goes through `red`, one word per wave.  Consecutive
// calls alternate between two halves of `red` (`turn`): a wave that runs
// ahead writes the other half, and the half it writes next is behind a
// barrier that every reader has passed.
template <int G>
__device__ __forceinline__ float row_sum(float v, float* red, int turn)
{
    v = wave_sum(v);
    if constexpr (G > 64) {
        float* r = red + (turn & 1) * (G / 64);
        if ((threadIdx.x & 63u) == 0) r[threadIdx.x >> 6] = v;
        __syncthreads();
        v = r[0];
#pragma unroll
        for (int w = 1; w < G / 64; ++w) v += r[w];
    }
    return v;
}
// two sums at once (`red`: two words per wave and turn)
template <int G>
__device__ __forceinline__ void row_sum2(float& v, float& w, float* red, int turn)
{
    v = wave_sum(v);
    w = wave_sum(w);
    if constexpr (G > 64) {
        float* r = red + (turn & 1) * (2 * G / 64);
        if ((threadIdx.x & 63u) == 0) *(f32x2*)(r + 2 * (threadIdx.x >> 6)) = f32x2{v, w};
        __syncthreads();
        f32x2 s = *(const f32x2*)r;
#pragma unroll
        for (int k = 1; k < G / 64; ++k) s += *(const f32x2*)(r + 2 * k);
        v = s.x;
        w = s.y;
    }
}
template <int G>
__device__ __forceinline__ uint32_t row_max_u32(uint32_t v, float* red, int turn)
{
    v = wave_max_u32(v);
    if constexpr (G > 64) {
        uint32_t* r = (uint32_t*)red + (turn & 1) * (G / 64);
        if ((threadIdx.x & 63u) == 0) r[threadIdx.x >> 6] = v;
        __syncthreads();
        v = r[0];
#pragma unroll
        for (int w = 1; w < G / 64; ++w) v = max(v, r[w]);
    }
    return v;
}

// threads of a row kernel's block: four rows of a wave each, or one row (whose
// reductions are barriers of the block)
template <int G>
constexpr int row_block() { return G == 64 ? 256 : G; }

}  // namespace echo
