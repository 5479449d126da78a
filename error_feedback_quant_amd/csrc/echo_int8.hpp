// echo_int8.hpp — gfx950 kernels of the 8-bit linear layer: token
// quantization and the integer product with a scale for each token and each
// channel.
//
// Quantization of a token x[0..K): a = max(max |x|, 2^-100), s = a / 127,
// q = rint(x * (127 / a)), all single IEEE fp32 operations.  |q| <= 127
// without a clamp: |x| * (127 / a) is at most 127 (1 + 2^-23).  A token that
// holds an infinity or a NaN gets the scale NaN and codes 0, so every output
// of that token is NaN rather than a plausible number.
//
// Product: y[m][n] = float(sum_k xq[m][k] wq[n][k]) * sx[m] * sw[n] + bias[n].
// The sum is exact in int32 for K <= 131071 (every product is at most 2^14 in
// magnitude), so neither its order nor the split of K can change a result.
// Rounding: the sum to fp32 (nearest even), each product, the bias sum, and
// once more to bf16 where y is bf16.
#pragma once

#include "echo_kernels.hpp"

namespace echo {

constexpr int kI8MaxK = (1 << 17) - 1;       // 2^14 * K stays below 2^31
constexpr float kI8Tiny = 0x1p-100f;         // smallest token magnitude that sets a scale

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

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

__device__ __forceinline__ float ld_elem(const void* p, bool bf16, int64_t i)
{
    return bf16 ? __builtin_bit_cast(float, (uint32_t)((const uint16_t*)p)[i] << 16) : ((const float*)p)[i];
}
__device__ __forceinline__ void st_elem(void* p, bool bf16, int64_t i, float v)
{
    if (bf16) ((uint16_t*)p)[i] = __builtin_bit_cast(uint16_t, (__bf16)v);
    else ((float*)p)[i] = v;
}

// Largest value over the block; every thread gets it.  red: one word per wave.
__device__ __forceinline__ uint32_t block_max_u32(uint32_t v, uint32_t* red)
{
#pragma unroll
    for (int o = 32; o; o >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o));
    if ((threadIdx.x & 63u) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
    for (uint32_t w = 1; w < blockDim.x / 64; ++w) v = max(v, red[w]);
    __syncthreads();
    return v;
}

struct QuantTokArgs {
    const void* x;
    int8_t* q;
    float* scale;
    int64_t ldx, ldq, T;
    int K;
    int bf16;
};

// One block per token, two passes over it.
__global__ __launch_bounds__(kBlock) void quantize_tokens_kernel(const QuantTokArgs a)
{
    __shared__ uint32_t red[kBlock / 64];
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        uint32_t m = 0;
        for (int k = threadIdx.x; k < a.K; k += kBlock) m = max(m, abs_bits(ld_elem(a.x, a.bf16, t * a.ldx + k)));
        const TokenScale s = token_scale(block_max_u32(m, red));
        for (int k = threadIdx.x; k < a.K; k += kBlock)
            a.q[t * a.ldq + k] = (int8_t)token_code(ld_elem(a.x, a.bf16, t * a.ldx + k), s.inv);
        if (threadIdx.x == 0) a.scale[t] = s.scale;
    }
}

struct GemmI8Args {
    const int8_t* x;        // [M] rows of ldx
    const int8_t* w;        // [N] rows of ldw
    const float* sx;        // [M]
    const float* sw;        // [N]
    const float* bias;      // [N], nullable
    void* y;                // [M] rows of ldy
    int64_t M, N, ldx, ldw, ldy;
    int K;
    int bf16;
    uint32_t tiles_m, tiles_n;
};

// 16 codes of a row from k on, zeros at and past K.  Only bytes below K are
// read: the last row of an operand may end where its allocation ends.  The
// address has any alignment (gfx950 loads 16 unaligned bytes in one access).
__device__ __forceinline__ i32x4 ld_codes16(const int8_t* row, int k, int K)
{
    i32x4 v = {0, 0, 0, 0};
    if (k + 16 <= K) {
        __builtin_memcpy(&v, row + k, 16);
    } else if (k < K) {
        for (int i = 0; i < K - k; ++i) {
            const uint32_t b = (uint32_t)(uint8_t)row[k + i] << (8 * (i & 3));
            const int d = i >> 2;
            v.x |= d == 0 ? b : 0u; v.y |= d == 1 ? b : 0u; v.z |= d == 2 ? b : 0u; v.w |= d == 3 ? b : 0u;
        }
    }
    return v;
}

__device__ __forceinline__ float gemm_i8_value(int acc, float sx, float sw, bool has_bias, float bias)
{
    const float y = ((float)acc * sx) * sw;
    return has_bias ? y + bias : y;
}

// A 64 x 64 output tile per 256-thread block: four waves of 32 x 32, K in
// steps of 64 bytes through registers into LDS.
__global__ __launch_bounds__(kBlock) void gemm_i8_tile_kernel(const GemmI8Args a)
{
    constexpr int kT = 64, kBK = 64;
    __shared__ __align__(16) i32x4 sx[kT][kBK / 16 + 1], sw[kT][kBK / 16 + 1];
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = tid >> 6;
    for (uint32_t tile = blockIdx.x; tile < a.tiles_m * a.tiles_n; tile += gridDim.x) {
        const int64_t m0 = (int64_t)(tile / a.tiles_n) * kT, n0 = (int64_t)(tile % a.tiles_n) * kT;
        const uint32_t r = tid >> 2, c = tid & 3u;
        const int8_t* xr = a.x + min(m0 + r, a.M - 1) * a.ldx;
        const int8_t* wr = a.w + min(n0 + r, a.N - 1) * a.ldw;
        i32x16 acc = {};
        for (int k0 = 0; k0 < a.K; k0 += kBK) {
            const i32x4 vx = ld_codes16(xr, k0 + 16 * c, a.K), vw = ld_codes16(wr, k0 + 16 * c, a.K);
            __syncthreads();
            sx[r][c] = vx;
            sw[r][c] = vw;
            __syncthreads();
#pragma unroll
            for (int kk = 0; kk < kBK / 32; ++kk) {
                const i32x4 fw = sw[(wave & 1u) * 32 + (lane & 31u)][2 * kk + (lane >> 5)];
                const i32x4 fx = sx[(wave >> 1) * 32 + (lane & 31u)][2 * kk + (lane >> 5)];
                acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw, fx, acc, 0, 0, 0);
            }
        }
        const int64_t m = m0 + (wave >> 1) * 32 + (lane & 31u);
        if (m < a.M) {
#pragma unroll
            for (int v = 0; v < 16; ++v) {
                const int64_t n = n0 + (wave & 1u) * 32 + 8 * (v >> 2) + 4 * (lane >> 5) + (v & 3);
                if (n < a.N)
                    st_elem(a.y, a.bf16, m * a.ldy + n,
                            gemm_i8_value(acc[v], a.sx[m], a.sw[n], a.bias, a.bias ? a.bias[n] : 0.0f));
            }
        }
    }
}

}  // namespace echo
