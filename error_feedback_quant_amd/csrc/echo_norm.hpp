// echo_norm.hpp — gfx950 kernels of the norms that close one block and open
// the next, around the gated, scaled residual sum, forward and backward.
//
//   k_x = rsqrt(mean x^2 + eps)             n_x = x k_x      (post norm)
//   z   = n_x w_post   (z = x without the post norm)
//   r'  = rho r + beta g z                  k_r = rsqrt(mean r'^2 + eps)
//   n_r = r' k_r                            h = n_r w_pre    (pre norm)
//
// Backward, from dh and dr' (recomputing k_x, k_r and r' from x and r, which
// the caller still holds, so nothing has to be saved between the passes and
// r' enters unrounded):
//   d     = dr' + k_r (dh w_pre - n_r mean(dh w_pre n_r))
//   dr    = rho d                           dw_pre  = sum_t dh n_r
//   dgate = sum over the gate's tokens of beta d z
//   dz    = beta g d                        dw_post = sum_t dz n_x
//   dx    = k_x (dz w_post - n_x mean(dz w_post n_x))
//
// Everything is held in fp32 and rounded once on its way out; h is computed
// from the unrounded r', and 8-bit codes of h from the unrounded h.
#pragma once

#include "echo_int8.hpp"

namespace echo {

struct NormArgs {
    const void* x;          // [T] rows of ld_x
    const void* r;          // [T] rows of ld_r, nullable (zero)
    const void* w_post;     // [H], nullable (ones)
    const void* w_pre;      // [H], nullable (ones)
    const void* gate;       // rows of ld_gate, one for gate_tokens tokens, nullable (ones)
    void* r_out;            // nullable
    void* h;                // nullable
    float* h_scale;         // [T], 8-bit h only
    int64_t T, ld_x, ld_r, ld_r_out, ld_h, ld_gate;
    uint32_t gate_tokens;   // at most T
    int H;
    int x_bf16, r_bf16, w_bf16, h_kind;    // h_kind: an echo_dtype
    int post;
    float eps, rho, beta;
};

struct NormBwdArgs {
    NormArgs f;
    const void* dh;         // nullable (zero)
    const void* dr_out;     // nullable (zero), type of r
    void* dx;               // nullable, type of x
    void* dr;               // nullable, type of r
    float* dw_post;
    float* dw_pre;
    float* dgate;
    int64_t ld_dh, ld_dr_out, ld_dx, ld_dr, ld_dgate;
    int dh_bf16;
    float* stats;           // [T][4]: k_x, k_r, mean(dh w_pre n_r), mean(dz w_post n_x)
    float* part;            // [chunks][2][H] partial dw_post, dw_pre
    int chunks;
};

__device__ __forceinline__ float block_sum(float v, float* red)
{
#pragma unroll
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    if ((threadIdx.x & 63u) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
    for (uint32_t w = 0; w < blockDim.x / 64; ++w) v += red[w];
    __syncthreads();
    return v;
}

__device__ __forceinline__ float norm_factor(float sum_sq, int H, float eps)
{
    return 1.0f / __builtin_sqrtf(sum_sq / (float)H + eps);
}

// one element's place in the formulas
struct NormElem {
    float x, n_x, w_post, z, g, r;
};
__device__ __forceinline__ NormElem norm_elem(const NormArgs& a, int64_t t, int c, float kx)
{
    NormElem e;
    e.x = ld_elem(a.x, a.x_bf16, t * a.ld_x + c);
    e.n_x = e.x * kx;
    e.w_post = a.w_post ? ld_elem(a.w_post, a.w_bf16, c) : 1.0f;
    e.z = a.post ? e.n_x * e.w_post : e.x;
    e.g = a.gate ? ld_elem(a.gate, a.w_bf16, (int64_t)((uint32_t)t / a.gate_tokens) * a.ld_gate + c) : 1.0f;
    const float r = a.r ? ld_elem(a.r, a.r_bf16, t * a.ld_r + c) : 0.0f;
    e.r = a.rho * r + a.beta * (e.g * e.z);
    return e;
}

// 8 weights (or gate values) of a row from k on; ones where there are none
template <bool TAIL>
__device__ __forceinline__ void ld_weights8(const void* base, int bf16, int64_t row, int k, int H, float (&w)[8])
{
    if (!base) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.0f;
    } else if (bf16) {
        const Raw8<true> r = ld_raw8<true, TAIL>(base, row, k, H);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = raw_get(r, e);
    } else {
        const Raw8<false> r = ld_raw8<false, TAIL>(base, row, k, H);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = raw_get(r, e);
    }
}

// A token held in registers: G threads, C chunks of 8 elements each, every
// byte moved once.  The weights stay in registers over the tokens of a group
// of threads, and so does the gate while its row lasts.
template <int G, int C, bool XB, bool RB, bool TAIL>
__global__ __launch_bounds__(row_block<G>()) void block_norm_kernel(const NormArgs a)
{
    __shared__ float red[G > 64 ? 2 * G / 64 : 1];
    constexpr int kRows = row_block<G>() / G;
    const int g = threadIdx.x % G;
    int64_t t = (int64_t)blockIdx.x * kRows + threadIdx.x / G;
    if constexpr (G == 64) t = __builtin_amdgcn_readfirstlane((int)t);
    const int64_t step = (int64_t)gridDim.x * kRows;
    float w_post[C][8], w_pre[C][8], gate[C][8];
#pragma unroll
    for (int j = 0; j < C; ++j) {
        ld_weights8<TAIL>(a.w_post, a.w_bf16, 0, 8 * (g + G * j), a.H, w_post[j]);
        ld_weights8<TAIL>(a.w_pre, a.w_bf16, 0, 8 * (g + G * j), a.H, w_pre[j]);
        ld_weights8<TAIL>(nullptr, 0, 0, 0, 0, gate[j]);
    }
    uint32_t gate_row = ~0u;
    int turn = 0;
    for (; t < a.T; t += step) {
        Raw8<XB> x[C];
        Raw8<RB> r[C];
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int k = 8 * (g + G * j);
            x[j] = ld_raw8<XB, TAIL>(a.x, t * a.ld_x, k, a.H);
            r[j] = ld_raw8<RB, TAIL>(a.r, t * a.ld_r, k, a.r ? a.H : 0);
        }
        if (a.gate) {
            const uint32_t row = (uint32_t)t / a.gate_tokens;
            if (row != gate_row) {
#pragma unroll
                for (int j = 0; j < C; ++j)
                    ld_weights8<TAIL>(a.gate, a.w_bf16, (int64_t)row * a.ld_gate, 8 * (g + G * j), a.H, gate[j]);
                gate_row = row;
            }
        }
        float kx = 1.0f;
        if (a.post) {
            float s = 0.0f;
#pragma unroll
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) s = fmaf(raw_get(x[j], e), raw_get(x[j], e), s);
            kx = norm_factor(row_sum<G>(s, red, turn++), a.H, a.eps);
        }
        float v[C][8];
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < C; ++j) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float z = raw_get(x[j], e) * kx * w_post[j][e];
                v[j][e] = a.rho * raw_get(r[j], e) + a.beta * (gate[j][e] * z);
                s = fmaf(v[j][e], v[j][e], s);
            }
            if (a.r_out) st_row8<RB, TAIL>(a.r_out, t * a.ld_r_out, 8 * (g + G * j), a.H, v[j]);
        }
        if (!a.h) continue;
        const float kr = norm_factor(row_sum<G>(s, red, turn++), a.H, a.eps);
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = v[j][e] * kr * w_pre[j][e];
        if (a.h_kind == ECHO_I8) {
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (!TAIL || 8 * (g + G * j) + e < a.H) m = max(m, abs_bits(v[j][e]));
            const TokenScale q = token_scale(row_max_u32<G>(m, red, turn++));
            if (g == 0) a.h_scale[t] = q.scale;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                int c[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) c[e] = token_code(v[j][e], q.inv);
                st_codes8<TAIL>((int8_t*)a.h, t * a.ld_h, 8 * (g + G * j), a.H, c);
            }
        } else if (a.h_kind == ECHO_BF16) {
#pragma unroll
            for (int j = 0; j < C; ++j) st_row8<true, TAIL>(a.h, t * a.ld_h, 8 * (g + G * j), a.H, v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < C; ++j) st_row8<false, TAIL>(a.h, t * a.ld_h, 8 * (g + G * j), a.H, v[j]);
        }
    }
}

// One block per token of any width; the row is read again in each pass.
__global__ __launch_bounds__(kBlock) void block_norm_any_kernel(const NormArgs a)
{
    __shared__ float red[kBlock / 64];
    __shared__ uint32_t redu[kBlock / 64];
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        float kx = 0.0f;
        if (a.post) {
            float s = 0.0f;
            for (int c = threadIdx.x; c < a.H; c += kBlock) {
                const float v = ld_elem(a.x, a.x_bf16, t * a.ld_x + c);
                s = fmaf(v, v, s);
            }
            kx = norm_factor(block_sum(s, red), a.H, a.eps);
        }
        float kr = 0.0f;
        TokenScale q = {0.0f, 0.0f};
        if (a.h) {
            float s = 0.0f;
            for (int c = threadIdx.x; c < a.H; c += kBlock) {
                const float v = norm_elem(a, t, c, kx).r;
                s = fmaf(v, v, s);
            }
            kr = norm_factor(block_sum(s, red), a.H, a.eps);
            if (a.h_kind == ECHO_I8) {
                uint32_t m = 0;
                for (int c = threadIdx.x; c < a.H; c += kBlock) {
                    const float w = a.w_pre ? ld_elem(a.w_pre, a.w_bf16, c) : 1.0f;
                    m = max(m, abs_bits(norm_elem(a, t, c, kx).r * kr * w));
                }
                q = token_scale(block_max_u32(m, redu));
                if (threadIdx.x == 0) a.h_scale[t] = q.scale;
            }
        }
        // r_out may be r: a column is read by the thread that writes it, and
        // the passes above are behind a barrier
        for (int c = threadIdx.x; c < a.H; c += kBlock) {
            const float v = norm_elem(a, t, c, kx).r;
            if (a.h) {
                const float h = v * kr * (a.w_pre ? ld_elem(a.w_pre, a.w_bf16, c) : 1.0f);
                if (a.h_kind == ECHO_I8) ((int8_t*)a.h)[t * a.ld_h + c] = (int8_t)token_code(h, q.inv);
                else st_elem(a.h, a.h_kind == ECHO_BF16, t * a.ld_h + c, h);
            }
            if (a.r_out) st_elem(a.r_out, a.r_bf16, t * a.ld_r_out + c, v);
        }
    }
}

// ---------------------------------------------------------------- backward --

struct NormGrad {
    NormElem e;
    float n_r, dh, dhw, d, dz;
};
// m: mean(dh w_pre n_r) (0 while it is being summed)
__device__ __forceinline__ NormGrad norm_grad(const NormBwdArgs& b, int64_t t, int c, float kx, float kr, float m)
{
    const NormArgs& a = b.f;
    NormGrad g;
    g.e = norm_elem(a, t, c, kx);
    g.n_r = g.e.r * kr;
    g.dh = b.dh ? ld_elem(b.dh, b.dh_bf16, t * b.ld_dh + c) : 0.0f;
    g.dhw = g.dh * (a.w_pre ? ld_elem(a.w_pre, a.w_bf16, c) : 1.0f);
    const float up = b.dr_out ? ld_elem(b.dr_out, a.r_bf16, t * b.ld_dr_out + c) : 0.0f;
    g.d = up + kr * (g.dhw - g.n_r * m);
    g.dz = a.beta * g.e.g * g.d;
    return g;
}

// the four numbers of a token that its gradients need
__global__ __launch_bounds__(kBlock) void norm_bwd_stats_kernel(const NormBwdArgs b)
{
    __shared__ float red[kBlock / 64];
    const NormArgs& a = b.f;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        float s = 0.0f;
        for (int c = threadIdx.x; c < a.H; c += kBlock) {
            const float v = ld_elem(a.x, a.x_bf16, t * a.ld_x + c);
            s = fmaf(v, v, s);
        }
        const float kx = norm_factor(block_sum(s, red), a.H, a.eps);
        s = 0.0f;
        for (int c = threadIdx.x; c < a.H; c += kBlock) {
            const float v = norm_elem(a, t, c, kx).r;
            s = fmaf(v, v, s);
        }
        const float kr = norm_factor(block_sum(s, red), a.H, a.eps);
        s = 0.0f;
        for (int c = threadIdx.x; c < a.H; c += kBlock) {
            const NormGrad g = norm_grad(b, t, c, kx, kr, 0.0f);
            s = fmaf(g.dhw, g.n_r, s);
        }
        const float m = block_sum(s, red) / (float)a.H;
        s = 0.0f;
        for (int c = threadIdx.x; c < a.H; c += kBlock) {
            const NormGrad g = norm_grad(b, t, c, kx, kr, m);
            s = fmaf(g.dz * g.e.w_post, g.e.n_x, s);
        }
        const float mx = block_sum(s, red) / (float)a.H;
        if (threadIdx.x == 0) *(f32x4*)(b.stats + 4 * t) = f32x4{kx, kr, m, mx};
    }
}

// partial weight gradients: one column per thread, one chunk of tokens per blockIdx.y
__global__ __launch_bounds__(kBlock) void norm_bwd_weights_kernel(const NormBwdArgs b)
{
    const NormArgs& a = b.f;
    const int c = blockIdx.x * kBlock + threadIdx.x;
    if (c >= a.H) return;
    const int64_t per = (a.T + b.chunks - 1) / b.chunks;
    const int64_t t1 = min(a.T, (blockIdx.y + 1) * per);
    float post = 0.0f, pre = 0.0f;
    for (int64_t t = blockIdx.y * per; t < t1; ++t) {
        const f32x4 s = *(const f32x4*)(b.stats + 4 * t);
        const NormGrad g = norm_grad(b, t, c, s.x, s.y, s.z);
        post += g.dz * g.e.n_x;
        pre += g.dh * g.n_r;
    }
    b.part[(int64_t)(2 * blockIdx.y) * a.H + c] = post;
    b.part[(int64_t)(2 * blockIdx.y + 1) * a.H + c] = pre;
}

__global__ __launch_bounds__(kBlock) void norm_bwd_weights_sum_kernel(const NormBwdArgs b)
{
    const int c = blockIdx.x * kBlock + threadIdx.x;
    if (c >= b.f.H) return;
    float post = 0.0f, pre = 0.0f;
    for (int k = 0; k < b.chunks; ++k) {
        post += b.part[(int64_t)(2 * k) * b.f.H + c];
        pre += b.part[(int64_t)(2 * k + 1) * b.f.H + c];
    }
    if (b.dw_post) b.dw_post[c] = post;
    if (b.dw_pre) b.dw_pre[c] = pre;
}

// a gate row's gradient: one column per thread, gate rows along blockIdx.y
__global__ __launch_bounds__(kBlock) void norm_bwd_gate_kernel(const NormBwdArgs b, int64_t rows)
{
    const NormArgs& a = b.f;
    const int c = blockIdx.x * kBlock + threadIdx.x;
    if (c >= a.H) return;
    for (int64_t g = blockIdx.y; g < rows; g += gridDim.y) {
        const int64_t t1 = min(a.T, (g + 1) * (int64_t)a.gate_tokens);
        float s = 0.0f;
        for (int64_t t = g * (int64_t)a.gate_tokens; t < t1; ++t) {
            const f32x4 st = *(const f32x4*)(b.stats + 4 * t);
            const NormGrad v = norm_grad(b, t, c, st.x, st.y, st.z);
            s += a.beta * v.d * v.e.z;
        }
        b.dgate[g * b.ld_dgate + c] = s;
    }
}

// dx and dr; dr may be dr_out
__global__ __launch_bounds__(kBlock) void norm_bwd_apply_kernel(const NormBwdArgs b)
{
    const NormArgs& a = b.f;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const f32x4 s = *(const f32x4*)(b.stats + 4 * t);
        for (int c = threadIdx.x; c < a.H; c += kBlock) {
            const NormGrad g = norm_grad(b, t, c, s.x, s.y, s.z);
            if (b.dr) st_elem(b.dr, a.r_bf16, t * b.ld_dr + c, a.rho * g.d);
            if (b.dx)
                st_elem(b.dx, a.x_bf16, t * b.ld_dx + c,
                        a.post ? s.x * (g.dz * g.e.w_post - g.e.n_x * s.w) : g.dz);
        }
    }
}

}  // namespace echo
