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
    float* stats;           // long rows: [T][4]: k_x, k_r, mean(dh w_pre n_r), mean(dz w_post n_x)
    float* part;            // [blocks or chunks][2][H] partial dw_post, dw_pre
    float* gpart;           // [groups][2][H] partial dgate of a group's first and last gate row
    int chunks;             // blocks of the row kernel, or chunks of tokens
    uint32_t per;           // tokens of a group
    uint32_t groups;        // groups that have tokens
    uint32_t spread;        // > 0: groups of a gate row (of all tokens without a gate), which go round its tokens
    uint32_t gate_rows;
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

// rsqrt(mean + eps) of a row from its sum of squares; 0 where that left fp32
__device__ __forceinline__ float norm_factor(float sum_sq, int H, float eps)
{
    return 1.0f / __builtin_sqrtf(sum_sq / (float)H + eps);
}
// Squares leave fp32 long before the values do (from about 2^64 / sqrt(H) on),
// and a factor of 0 would let the row vanish: such a row is summed again by
// `scaled_sum`, over its values times kNormSmall (2^30 squares of 2^48 at the
// most).  A row that holds an infinity or a NaN has the factor NaN, so that
// none of its normed values passes for a number.
constexpr float kNormSmall = 0x1p-80f;
template <typename F>
__device__ __forceinline__ float norm_factor(float sum_sq, int H, float eps, F scaled_sum)
{
    if (__builtin_expect(sum_sq / (float)H + eps < __builtin_inff(), 1)) return norm_factor(sum_sq, H, eps);
    const float m = scaled_sum() / (float)H + eps * kNormSmall * kNormSmall;
    return m < __builtin_inff() ? kNormSmall / __builtin_sqrtf(m) : __builtin_nanf("");
}
// Backward, tokens with a smaller factor than this take a way of their own: a
// product of three factors, or a sum of values times gradients, may leave
// fp32 where the results do not.
constexpr float kNormLeast = 0x1p-40f;

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

// beta gate w_post of 8 columns, what a normed x is multiplied by
template <bool TAIL>
__device__ __forceinline__ void ld_branch8(const NormArgs& a, const void* gate, int64_t row, int k, float (&w)[8])
{
    float g[8];
    ld_weights8<TAIL>(a.w_post, a.w_bf16, 0, k, a.H, w);
    ld_weights8<TAIL>(gate, a.w_bf16, row, k, a.H, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = a.beta * g[e] * w[e];
}

// A token held in registers: G threads, C chunks of 8 elements each, every
// byte moved once.  The weights stay in registers over the tokens of a group
// of threads, and so does the gate while its row lasts.  Bound by memory:
// 131072 x 1024 in bf16 (1.07 GB) takes 182 us, 5.9 TB/s (a device copy
// reaches 4.9); 2048 x 4096 with an fp32 stream and gate (100 MB) 23 us; 64 x
// 1024 is 4.2 us of load, two reductions and store after one another.
template <int G, int C, bool XB, bool RB, bool TAIL>
__global__ __launch_bounds__(row_block<G>()) void block_norm_kernel(const NormArgs a)
{
    __shared__ float red[G > 64 ? 2 * G / 64 : 1];
    constexpr int kRows = row_block<G>() / G;
    const int g = threadIdx.x % G;
    int64_t t = (int64_t)blockIdx.x * kRows + threadIdx.x / G;
    t = __builtin_amdgcn_readfirstlane((int)t);              // one row a wave at most: kept in scalar registers
    const int64_t step = (int64_t)gridDim.x * kRows;
    float w[C][8], w_pre[C][8];                              // w: beta gate w_post
    auto weights = [&](const void* gate, int64_t row) {
#pragma unroll
        for (int j = 0; j < C; ++j) ld_branch8<TAIL>(a, gate, row, 8 * (g + G * j), w[j]);
    };
    weights(nullptr, 0);
#pragma unroll
    for (int j = 0; j < C; ++j) ld_weights8<TAIL>(a.w_pre, a.w_bf16, 0, 8 * (g + G * j), a.H, w_pre[j]);
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
            if (row != gate_row) weights(a.gate, (int64_t)row * a.ld_gate);
            gate_row = row;
        }
        float kx = 1.0f;
        if (a.post) {
            float s = 0.0f;
#pragma unroll
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) s = fmaf(raw_get(x[j], e), raw_get(x[j], e), s);
            kx = norm_factor(row_sum<G>(s, red, turn++), a.H, a.eps, [&] {
                float b = 0.0f;
#pragma unroll
                for (int j = 0; j < C; ++j)
#pragma unroll
                    for (int e = 0; e < 8; ++e) b = fmaf(raw_get(x[j], e) * kNormSmall, raw_get(x[j], e) * kNormSmall, b);
                return row_sum<G>(b, red, turn++);
            });
        }
        float v[C][8];
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < C; ++j) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[j][e] = fmaf(raw_get(x[j], e) * kx, w[j][e], a.rho * raw_get(r[j], e));
                s = fmaf(v[j][e], v[j][e], s);
            }
            if (a.r_out) st_row8<RB, TAIL>(a.r_out, t * a.ld_r_out, 8 * (g + G * j), a.H, v[j]);
        }
        if (!a.h) continue;
        const float kr = norm_factor(row_sum<G>(s, red, turn++), a.H, a.eps, [&] {
            float b = 0.0f;
#pragma unroll
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) b = fmaf(v[j][e] * kNormSmall, v[j][e] * kNormSmall, b);
            return row_sum<G>(b, red, turn++);
        });
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

// Factor of a row that a block walks over: value(c) is its element c
template <typename F>
__device__ __forceinline__ float row_factor(const NormArgs& a, float* red, F value)
{
    auto sum = [&](float scale) {
        float s = 0.0f;
        for (int c = threadIdx.x; c < a.H; c += kBlock) {
            const float v = value(c) * scale;
            s = fmaf(v, v, s);
        }
        return block_sum(s, red);
    };
    return norm_factor(sum(1.0f), a.H, a.eps, [&] { return sum(kNormSmall); });
}

// Rows too wide for registers: one block per token of any width, the row read
// again in each pass (from L2 where it fits).  Single elements a lane and
// load, so far from memory's rate: 2048 x 20000 in bf16 (328 MB) takes 355 us.
__global__ __launch_bounds__(kBlock) void block_norm_any_kernel(const NormArgs a)
{
    __shared__ float red[kBlock / 64];
    __shared__ uint32_t redu[kBlock / 64];
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        float kx = 0.0f;
        if (a.post) kx = row_factor(a, red, [&](int c) { return ld_elem(a.x, a.x_bf16, t * a.ld_x + c); });
        float kr = 0.0f;
        TokenScale q = {0.0f, 0.0f};
        if (a.h) {
            kr = row_factor(a, red, [&](int c) { return norm_elem(a, t, c, kx).r; });
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

// Backward of rows too wide for registers (over 8192 elements), in passes that
// read them again: each token's four numbers, the sums over tokens by columns,
// then dx and dr.  Each pass loads single elements, so far from memory's rate:
// 2048 x 12288 in bf16 (302 MB) takes 642 us, 3.3 ms with one gate row for all
// tokens, where one thread walks a column.

// the four numbers of a token that its gradients need
__global__ __launch_bounds__(kBlock) void norm_bwd_stats_kernel(const NormBwdArgs b)
{
    __shared__ float red[kBlock / 64];
    const NormArgs& a = b.f;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const float kx = row_factor(a, red, [&](int c) { return ld_elem(a.x, a.x_bf16, t * a.ld_x + c); });
        const float kr = row_factor(a, red, [&](int c) { return norm_elem(a, t, c, kx).r; });
        float s = 0.0f;
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
    const int64_t per = (a.T + b.chunks - 1) / b.chunks;   // chunks > 0: there are tokens
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
__global__ __launch_bounds__(kBlock) void norm_bwd_gate_kernel(const NormBwdArgs b)
{
    const NormArgs& a = b.f;
    const int c = blockIdx.x * kBlock + threadIdx.x;
    if (c >= a.H) return;
    for (int64_t g = blockIdx.y; g < b.gate_rows; g += gridDim.y) {
        const int64_t t1 = min(a.T, (g + 1) * (int64_t)a.gate_tokens);
        // a chain as long as the gate row: the rounding of each addition is
        // carried to the next (60000 equal tokens: off by 1e-3 without, 1e-7 with)
        float s = 0.0f, lost = 0.0f;
        for (int64_t t = g * (int64_t)a.gate_tokens; t < t1; ++t) {
            const f32x4 st = *(const f32x4*)(b.stats + 4 * t);
            const NormGrad v = norm_grad(b, t, c, st.x, st.y, st.z);
            const float add = a.beta * v.d * v.e.z - lost, sum = s + add;
            lost = (sum - s) - add;
            s = sum;
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

// Tokens held in registers, every row moved once.  A group of G threads takes
// `per` consecutive tokens and keeps its columns' sums in registers over them;
// the next token's rows are loaded before this one is worked on.
//
// Two sums for three gradients: with A = sum of d n_x over a gate row's tokens
// (n_x = x without the post norm), dgate = beta w_post A, and dw_post is the
// sum of beta gate A over the gate rows.
//
// Partial sums go to the workspace and norm_bwd_sum_kernel adds them in a
// fixed order, so equal inputs give equal bits:
//  * dw_post and dw_pre: the groups of a block meet in LDS, one partial a block;
//  * dgate: a gate row that lies inside one group's tokens is written at
//    once; one that a group shares with others goes to that group's slot 0
//    (its first gate row) or 1 (its last).  A block whose tokens all share
//    one gate row adds its groups up in LDS and uses its first slot only.
// Where each gate row can have whole blocks of its own, its tokens go round
// their groups instead of in runs.
// Three reductions a token: sum x^2; sum r'^2 with sum dh w_pre r'; and
// sum dz w_post x.
//
// Bound by memory: 131072 x 1024 in bf16 (1.61 GB) takes 303 us, 5.3 TB/s,
// its second launch included.  One chunk a thread: with two the sums, weights
// and two tokens' rows fill 256 registers and spill (333 to 341 us).  2048 x
// 4096 with gate rows of 600 tokens (151 MB) takes 42 us, 37 + 4.8: one block
// of 8 waves on a CU, 8 tokens after one another, three barriers each.
template <int G, int C, bool XB, bool RB, bool HB, bool TAIL>
__global__ __launch_bounds__(row_block<G>()) void block_norm_bwd_kernel(const NormBwdArgs b)
{
    constexpr int kGroups = row_block<G>() / G;
    __shared__ __align__(8) float red[G > 64 ? 6 * G / 64 : 2];
    __shared__ float meet[kGroups > 1 ? (kGroups - 1) * G * C * 8 : 1];
    const NormArgs& a = b.f;
    int g = threadIdx.x % G;
    const int q = threadIdx.x / G;
    const int64_t group = (int64_t)blockIdx.x * kGroups + q;
    uint32_t t0 = (uint32_t)min(a.T, group * b.per), t1 = (uint32_t)min(a.T, (group + 1) * b.per);
    if constexpr (G == 64) {
        t0 = __builtin_amdgcn_readfirstlane(t0);
        t1 = __builtin_amdgcn_readfirstlane(t1);
    }
    // Spread: neighbouring tokens go to neighbouring groups, each gate row to
    // groups of its own, so that the chip works on few stretches of memory at
    // a time (one without a gate).  A block's groups then share a gate row.
    const uint32_t step = b.spread ? b.spread : 1;
    if (b.spread) {
        const uint32_t span = a.gate ? a.gate_tokens : (uint32_t)a.T;
        const int64_t r0 = (group / b.spread) * (int64_t)span;
        t1 = (uint32_t)min(a.T, r0 + span);
        t0 = (uint32_t)min((int64_t)t1, r0 + group % b.spread);
    }
    const float invH = 1.0f / (float)a.H;
    float s_post[C][8], s_pre[C][8], sum[C][8], w[C][8], w_pre[C][8];   // w: beta gate w_post
    auto weights = [&](const void* gate, int64_t row) {
#pragma unroll
        for (int j = 0; j < C; ++j) ld_branch8<TAIL>(a, gate, row, 8 * (g + G * j), w[j]);
    };
    weights(nullptr, 0);
#pragma unroll
    for (int j = 0; j < C; ++j) {
        ld_weights8<TAIL>(a.w_pre, a.w_bf16, 0, 8 * (g + G * j), a.H, w_pre[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) s_post[j][e] = s_pre[j][e] = sum[j][e] = 0.0f;
    }
    // whole block on one gate row (its dgate is then left to the block's end)
    const uint32_t bt0 = (uint32_t)min(a.T, (int64_t)blockIdx.x * kGroups * b.per);
    const uint32_t bt1 = (uint32_t)min(a.T, ((int64_t)blockIdx.x + 1) * kGroups * b.per);
    const bool one_row = a.gate && (b.spread ? true : a.gate_tokens > 1 && bt1 > bt0 &&
                                                          bt0 / a.gate_tokens == (bt1 - 1) / a.gate_tokens);
    // dw_post takes up the sum of a gate row (or of all tokens), the sum becomes dgate
    auto close = [&](const void* gate, int64_t row, float (&sum)[C][8]) {
#pragma unroll
        for (int j = 0; j < C; ++j) {
            float v[8];
            ld_weights8<TAIL>(gate, a.w_bf16, row, 8 * (g + G * j), a.H, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) s_post[j][e] = fmaf(a.beta * v[e], sum[j][e], s_post[j][e]);
            ld_weights8<TAIL>(a.w_post, a.w_bf16, 0, 8 * (g + G * j), a.H, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[j][e] *= a.beta * v[e];
        }
    };
    auto put = [&](float* to, int64_t row, float (&v)[C][8]) {
#pragma unroll
        for (int j = 0; j < C; ++j) st_row8<false, TAIL>(to, row, 8 * (g + G * j), a.H, v[j]);
    };
    // the gate row that ends (for this group) at token `end`; f(array, row in it) stores its sum
    auto place = [&](uint32_t row, uint32_t end, auto f) {
        const uint64_t r0 = (uint64_t)row * a.gate_tokens;
        const bool whole = r0 >= t0 && (r0 + a.gate_tokens <= end || end == (uint32_t)a.T);
        if (whole) f(b.dgate, (int64_t)row * b.ld_dgate);
        else f(b.gpart, (2 * group + (r0 > t0 ? 1 : 0)) * (int64_t)a.H);
    };
    auto flush = [&](uint32_t row, uint32_t end) {
        close(a.gate, (int64_t)row * a.ld_gate, sum);
        if (b.dgate && !one_row) place(row, end, [&](float* to, int64_t at) { put(to, at, sum); });
    };

    Raw8<XB> x[C], nx[C];
    Raw8<RB> r[C], nr[C], up[C], nup[C];
    Raw8<HB> dh[C], ndh[C];
    auto load = [&](uint32_t t) {
#pragma unroll
        for (int j = 0; j < C; ++j) {
            const int k = 8 * (g + G * j);
            nx[j] = ld_raw8<XB, TAIL>(a.x, (int64_t)t * a.ld_x, k, a.H);
            nr[j] = ld_raw8<RB, TAIL>(a.r, (int64_t)t * a.ld_r, k, a.r ? a.H : 0);
            ndh[j] = ld_raw8<HB, TAIL>(b.dh, (int64_t)t * b.ld_dh, k, b.dh ? a.H : 0);
            nup[j] = ld_raw8<RB, TAIL>(b.dr_out, (int64_t)t * b.ld_dr_out, k, b.dr_out ? a.H : 0);
        }
    };
    uint32_t gate_row = ~0u;
    int turn = 0;
    bool far = false;
    if (t0 < t1) load(t0);
    for (uint32_t t = t0; t < t1; t += step) {
#pragma unroll
        for (int j = 0; j < C; ++j) { x[j] = nx[j]; r[j] = nr[j]; dh[j] = ndh[j]; up[j] = nup[j]; }
        if (a.gate) {
            const uint32_t row = t / a.gate_tokens;
            if (row != gate_row) {
                if (gate_row != ~0u) {
                    flush(gate_row, t);
#pragma unroll
                    for (int j = 0; j < C; ++j)
#pragma unroll
                        for (int e = 0; e < 8; ++e) sum[j][e] = 0.0f;
                }
                weights(a.gate, (int64_t)row * a.ld_gate);
                gate_row = row;
            }
        }
        if (t + step < t1) load(t + step);
        float kx = 1.0f;
        if (a.post) {
            float s = 0.0f;
#pragma unroll
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) s = fmaf(raw_get(x[j], e), raw_get(x[j], e), s);
            kx = norm_factor(row_sum<G>(s, red, turn++), a.H, a.eps);
        }
        float v[C][8];                                       // r', then d
        float s = 0.0f, p = 0.0f;
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[j][e] = fmaf(raw_get(x[j], e) * kx, w[j][e], a.rho * raw_get(r[j], e));
                s = fmaf(v[j][e], v[j][e], s);
                p = fmaf(raw_get(dh[j], e) * w_pre[j][e], v[j][e], p);
            }
        row_sum2<G>(s, p, red + (G > 64 ? 2 * G / 64 : 0), turn);
        ++turn;
        float kr = norm_factor(s, a.H, a.eps);
        // A token left to the loop below adds zeros here, with factors of 0,
        // and is not stored (a branch around the rest costs registers).
        const bool near = kx >= kNormLeast && kr >= kNormLeast;
        far |= !near;
        const float km = near ? p * kr * invH * kr : 0.0f;   // k_r mean(dh w_pre n_r)
        kx = near ? kx : 0.0f;
        kr = near ? kr : 0.0f;
        float o = 0.0f;
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float n = v[j][e] * kr, h = raw_get(dh[j], e), xe = raw_get(x[j], e);
                s_pre[j][e] = fmaf(h, n, s_pre[j][e]);
                v[j][e] = fmaf(-n, km, fmaf(kr, h * w_pre[j][e], raw_get(up[j], e)));
                sum[j][e] = fmaf(v[j][e], xe * kx, sum[j][e]);
                o = fmaf(v[j][e] * w[j][e], xe, o);
            }
        if (b.dr && near) {
#pragma unroll
            for (int j = 0; j < C; ++j) {
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = a.rho * v[j][e];
                st_row8<RB, TAIL>(b.dr, (int64_t)t * b.ld_dr, 8 * (g + G * j), a.H, y);
            }
        }
        if (b.dx && near) {
            float mx = 0.0f;                                 // k_x^2 mean(dz w_post n_x)
            if (a.post) mx = row_sum<G>(o, red, turn++) * kx * invH * kx * kx;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = fmaf(-raw_get(x[j], e), mx, kx * (v[j][e] * w[j][e]));
                st_row8<XB, TAIL>(b.dx, (int64_t)t * b.ld_dx, 8 * (g + G * j), a.H, y);
            }
        }
    }
    if (!a.gate) close(nullptr, 0, sum);
    else if (gate_row != ~0u) flush(gate_row, t1);

    // Tokens of values too large for the products above, or of some that are no
    // numbers: the same gradients from their normed values, added to the sums
    // above.  In a loop of its own after those are done, because in the loop
    // above it costs that one registers (8000 rows of 8192 in fp32: 492 us, 315
    // here).  g is made opaque at each use, or the addresses that both loops
    // work out of it are kept, and spilled, from the kernel's start on.
    if (far) {
        asm("" : "+v"(g));
        float more[C][8];
        auto clear = [&] {
#pragma unroll
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) more[j][e] = 0.0f;
        };
        auto join = [&](uint32_t row, uint32_t end) {
            close(a.gate, (int64_t)row * a.ld_gate, more);
            if (b.dgate && one_row) {
#pragma unroll
                for (int j = 0; j < C; ++j)
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum[j][e] += more[j][e];
            } else if (b.dgate) {
                place(row, end, [&](float* to, int64_t at) {
#pragma unroll
                    for (int j = 0; j < C; ++j) {
                        const Raw8<false> had = ld_raw8<false, TAIL>(to, at, 8 * (g + G * j), a.H);
#pragma unroll
                        for (int e = 0; e < 8; ++e) more[j][e] += raw_get(had, e);
                    }
                    put(to, at, more);
                });
            }
            clear();
        };
        clear();
        gate_row = ~0u;
        for (uint32_t t = t0; t < t1; t += step) {
            asm("" : "+v"(g));
            if (a.gate) {
                const uint32_t row = t / a.gate_tokens;
                if (row != gate_row) {
                    if (gate_row != ~0u) join(gate_row, t);
                    weights(a.gate, (int64_t)row * a.ld_gate);
                    gate_row = row;
                }
            }
            float v[C][8], kx = 1.0f, kr;
            // the loop's own factor, by which it left the token out, and the one that holds for large values
            auto factor = [&](auto value, float& k) {
                auto sum_sq = [&](float scale) {
                    float q = 0.0f, none = 0.0f;
#pragma unroll
                    for (int j = 0; j < C; ++j)
#pragma unroll
                        for (int e = 0; e < 8; ++e) q = fmaf(value(j, e) * scale, value(j, e) * scale, q);
                    row_sum2<G>(q, none, red + (G > 64 ? 2 * G / 64 : 0), turn++);
                    return q;
                };
                const float q = sum_sq(1.0f);
                k = norm_factor(q, a.H, a.eps, [&] { return sum_sq(kNormSmall); });
                return !(norm_factor(q, a.H, a.eps) >= kNormLeast);
            };
            bool is_far = false;
#pragma unroll
            for (int j = 0; j < C; ++j) x[j] = ld_raw8<XB, TAIL>(a.x, (int64_t)t * a.ld_x, 8 * (g + G * j), a.H);
            if (a.post) is_far = factor([&](int j, int e) { return raw_get(x[j], e); }, kx);
#pragma unroll
            for (int j = 0; j < C; ++j) {
                r[j] = ld_raw8<RB, TAIL>(a.r, (int64_t)t * a.ld_r, 8 * (g + G * j), a.r ? a.H : 0);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[j][e] = fmaf(raw_get(x[j], e) * kx, w[j][e], a.rho * raw_get(r[j], e));
            }
            is_far |= factor([&](int j, int e) { return v[j][e]; }, kr);
            if (!is_far) continue;
            float s = 0.0f;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                dh[j] = ld_raw8<HB, TAIL>(b.dh, (int64_t)t * b.ld_dh, 8 * (g + G * j), b.dh ? a.H : 0);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    v[j][e] *= kr;                           // n_r, then d
                    s = fmaf(raw_get(dh[j], e) * w_pre[j][e], v[j][e], s);
                }
            }
            const float m = row_sum<G>(s, red, turn++) * invH;
            s = 0.0f;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                float y[8];
                up[j] = ld_raw8<RB, TAIL>(b.dr_out, (int64_t)t * b.ld_dr_out, 8 * (g + G * j), b.dr_out ? a.H : 0);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float n = v[j][e], h = raw_get(dh[j], e), n_x = raw_get(x[j], e) * kx;
                    s_pre[j][e] = fmaf(h, n, s_pre[j][e]);
                    v[j][e] = fmaf(kr, fmaf(h, w_pre[j][e], -n * m), raw_get(up[j], e));
                    y[e] = a.rho * v[j][e];
                    more[j][e] = fmaf(v[j][e], n_x, more[j][e]);
                    v[j][e] *= w[j][e];
                    s = fmaf(v[j][e], n_x, s);
                }
                if (b.dr) st_row8<RB, TAIL>(b.dr, (int64_t)t * b.ld_dr, 8 * (g + G * j), a.H, y);
            }
            if (!b.dx) continue;
            const float mx = a.post ? row_sum<G>(s, red, turn++) * invH : 0.0f;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = kx * fmaf(-(raw_get(x[j], e) * kx), mx, v[j][e]);
                st_row8<XB, TAIL>(b.dx, (int64_t)t * b.ld_dx, 8 * (g + G * j), a.H, y);
            }
        }
        asm("" : "+v"(g));
        if (!a.gate) close(nullptr, 0, more);
        else join(gate_row, t1);
    }

    // sums of the block: group 0 adds the others' from LDS
    auto gather = [&](float (&v)[C][8]) {
        if constexpr (kGroups > 1) {
            if (q > 0) {
#pragma unroll
                for (int j = 0; j < C; ++j)
#pragma unroll
                    for (int e = 0; e < 8; ++e) meet[(((q - 1) * C + j) * 8 + e) * G + g] = v[j][e];
            }
            __syncthreads();
            if (q == 0) {
#pragma unroll
                for (int j = 0; j < C; ++j)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        for (int o = 0; o < kGroups - 1; ++o) v[j][e] += meet[((o * C + j) * 8 + e) * G + g];
            }
            __syncthreads();
        }
    };
    if (b.dgate && one_row) {
        gather(sum);
        if (q == 0) put(b.gpart, 2 * group * (int64_t)a.H, sum);
    }
    gather(s_post);
    gather(s_pre);
    if (q == 0) {
        put(b.part, (int64_t)(2 * blockIdx.x) * a.H, s_post);
        put(b.part, (int64_t)(2 * blockIdx.x + 1) * a.H, s_pre);
    }
}

// Adds the partial sums (bound by latency: 3.9 to 6.1 us for 167 to 1024
// partials): blockIdx.x a strip of 64 columns, blockIdx.y 0 and 1
// dw_post and dw_pre, from 2 on the gate rows.  16 waves share a column's
// partials and meet in LDS.
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(64 * kSumWaves) void norm_bwd_sum_kernel(const NormBwdArgs b, int group_shift)
{
    __shared__ float meet[kSumWaves][64];
    const NormArgs& a = b.f;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    auto finish = [&](float s, float* to) {
        meet[wave][lane] = s;
        __syncthreads();
        if (wave == 0 && c < a.H) {
#pragma unroll
            for (int w = 1; w < kSumWaves; ++w) s += meet[w][lane];
            *to = s;
        }
        __syncthreads();
    };
    if (blockIdx.y < 2) {
        float* to = blockIdx.y ? b.dw_pre : b.dw_post;
        if (!to) return;
        float s = 0.0f;
        if (c < a.H) {
#pragma unroll 8
            for (int k = wave; k < b.chunks; k += kSumWaves) s += b.part[(int64_t)(2 * k + blockIdx.y) * a.H + c];
        }
        finish(s, to + c);
        return;
    }
    if (b.spread) {                                          // each block's first slot holds its sum
        const uint32_t row = blockIdx.y - 2;
        float s = 0.0f;
        if (c < a.H) {
#pragma unroll 8
            for (uint32_t k = wave; k < b.spread >> group_shift; k += kSumWaves)
                s += b.gpart[2 * ((int64_t)row * b.spread + ((int64_t)k << group_shift)) * a.H + c];
        }
        finish(s, b.dgate + (int64_t)row * b.ld_dgate + c);
        return;
    }
    const uint32_t block_tokens = b.per << group_shift;      // 1 << group_shift groups a block
    // A row that is not written yet ends its first group (or goes past it),
    // so where there are more rows than groups it is found by the group.
    const bool by_row = b.gate_rows <= b.groups;
    const uint32_t n = by_row ? b.gate_rows : b.groups;
    for (uint32_t i = blockIdx.y - 2; i < n; i += gridDim.y - 2) {
        const uint32_t row = by_row ? i : ((uint32_t)min(a.T, (int64_t)(i + 1) * b.per) - 1) / a.gate_tokens;
        const uint32_t r0 = row * a.gate_tokens, r1 = (uint32_t)min(a.T, (int64_t)r0 + a.gate_tokens);
        const uint32_t q0 = r0 / b.per, q1 = (r1 - 1) / b.per;
        if (!by_row && q0 != i) continue;
        // a block that lies in the row has added up its groups (no division: they took half of this kernel's time)
        auto inside = [&](uint32_t block) {
            const uint32_t k0 = block * block_tokens;
            return k0 >= r0 && (uint32_t)min(a.T, (int64_t)k0 + block_tokens) <= r1;
        };
        // inside one group, in a block with other gate rows: already written
        if (q0 == q1 && !inside(q0 >> group_shift)) continue;
        float s = 0.0f;
        if (c < a.H) {
#pragma unroll 8
            for (uint32_t k = q0 + wave; k <= q1; k += kSumWaves) {
                const bool added = ((k >> group_shift) << group_shift) != k && inside(k >> group_shift);
                if (!added) s += b.gpart[(int64_t)(2 * k + (r0 > k * b.per ? 1 : 0)) * a.H + c];
            }
        }
        finish(s, b.dgate + (int64_t)row * b.ld_dgate + c);
    }
}

}  // namespace echo
