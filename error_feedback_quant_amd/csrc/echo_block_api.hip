// echo_block_api.hip — host side of the operators around the all-reduce of a
// tensor-parallel block: token quantization, the 8-bit product and linear
// layer, and the block norms.  Argument checks and launches; semantics,
// layouts and error behaviour are specified in include/echo.h.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "echo.h"
#include "echo_host.hpp"
#include "echo_int8.hpp"
#include "echo_norm.hpp"

namespace {

using echo::aligned16;
using echo::aligned_to;
using echo::check_launch;

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxLd = int64_t(1) << 32;        // row strides; offsets are 64-bit
constexpr int64_t kMaxGrid = int64_t(1) << 20;      // blocks of a launch; kernels stride over the rest

bool float_dtype(int d) { return d == ECHO_F32 || d == ECHO_BF16; }
size_t dtype_bytes(int d) { return d == ECHO_F32 ? 4 : (d == ECHO_BF16 ? 2 : 1); }
bool aligned_elem(const void* p, int dtype) { return aligned_to(p, dtype_bytes(dtype)); }

// rows of `cols` elements at a distance of ld (which a single row does not use)
bool bad_ld(int64_t ld, int64_t rows, int64_t cols) { return rows > 1 && (ld < cols || ld > kMaxLd); }
bool bad_dim(int64_t v, int64_t most) { return v < 0 || v > most; }

unsigned grid_of(int64_t items) { return (unsigned)(items < kMaxGrid ? items : kMaxGrid); }

void launch_quantize(const echo::QuantTokArgs& a, hipStream_t st)
{
    hipLaunchKernelGGL(echo::quantize_tokens_kernel, dim3(grid_of(a.T)), dim3(echo::kBlock), 0, st, a);
}

void launch_gemm_i8(echo::GemmI8Args& a, hipStream_t st)
{
    a.tiles_m = (uint32_t)((a.M + 63) / 64);
    a.tiles_n = (uint32_t)((a.N + 63) / 64);
    hipLaunchKernelGGL(echo::gemm_i8_tile_kernel, dim3(grid_of((int64_t)a.tiles_m * a.tiles_n)), dim3(echo::kBlock), 0,
                       st, a);
}

// the checks that echo_gemm_int8 and echo_linear_int8 share
int check_product(const int8_t* w, int64_t ldw, const float* sw, const float* bias, int64_t M, int64_t N, int64_t K,
                  const void* y, int64_t ldy, int y_dtype)
{
    if (!float_dtype(y_dtype)) return ECHO_EUNSUP;
    if (bad_dim(M, kMaxRows) || bad_dim(N, kMaxRows) || bad_dim(K, echo::kI8MaxK)) return ECHO_ESHAPE;
    if (bad_ld(ldw, N, K) || bad_ld(ldy, M, N)) return ECHO_ESHAPE;
    if ((M + 63) / 64 * ((N + 63) / 64) > kMaxRows) return ECHO_ESHAPE;
    if (M == 0 || N == 0) return ECHO_OK;
    if ((K && !w) || !sw || !y) return ECHO_EINVAL;
    if (!aligned_to(sw, 4) || (bias && !aligned_to(bias, 4)) || !aligned_elem(y, y_dtype)) return ECHO_EALIGN;
    return ECHO_OK;
}

echo::GemmI8Args gemm_args(const int8_t* x, int64_t ldx, const float* sx, const int8_t* w, int64_t ldw, const float* sw,
                           const float* bias, int64_t M, int64_t N, int64_t K, void* y, int64_t ldy, int y_dtype)
{
    echo::GemmI8Args a;
    std::memset(&a, 0, sizeof(a));
    a.x = x; a.w = w; a.sx = sx; a.sw = sw; a.bias = bias; a.y = y;
    a.M = M; a.N = N; a.ldx = ldx; a.ldw = ldw; a.ldy = ldy;
    a.K = (int)K; a.bf16 = y_dtype == ECHO_BF16;
    return a;
}

// codes of the linear layer's tokens: rows of a multiple of 16, then the scales
int64_t codes_ld(int64_t K) { return (K + 15) / 16 * 16; }

// ------------------------------------------------------------------ norms --

constexpr int64_t kMaxWidth = int64_t(1) << 30;
constexpr int64_t kMaxChunks = 256;

int norm_chunks(int64_t T) { return (int)(T / 16 < 1 ? 1 : (T / 16 > kMaxChunks ? kMaxChunks : T / 16)); }

size_t norm_stats_bytes(int64_t T) { return (size_t)(T * 16); }

int check_norm(const echo_norm_args* p, bool backward)
{
    if (!p) return ECHO_EINVAL;
    const echo_norm_args& a = *p;
    if (!float_dtype(a.x_dtype) || !float_dtype(a.r_dtype) || !float_dtype(a.w_dtype)) return ECHO_EUNSUP;
    if (!backward && a.h && !float_dtype(a.h_dtype) && a.h_dtype != ECHO_I8) return ECHO_EUNSUP;
    if (bad_dim(a.T, kMaxRows) || bad_dim(a.H, kMaxWidth)) return ECHO_ESHAPE;
    if (bad_ld(a.ld_x, a.T, a.H) || (a.r && bad_ld(a.ld_r, a.T, a.H))) return ECHO_ESHAPE;
    if (!backward && ((a.r_out && bad_ld(a.ld_r_out, a.T, a.H)) || (a.h && bad_ld(a.ld_h, a.T, a.H))))
        return ECHO_ESHAPE;
    if (a.post != 0 && a.post != 1) return ECHO_EINVAL;
    if (!(a.eps > 0.0f) || !std::isfinite(a.eps) || !std::isfinite(a.res_scale) || !std::isfinite(a.block_scale))
        return ECHO_EINVAL;
    if (!a.post && a.w_post) return ECHO_EINVAL;
    if (a.gate) {
        if (a.gate_tokens < 1) return ECHO_EINVAL;
        if (bad_ld(a.ld_gate, (a.T + a.gate_tokens - 1) / a.gate_tokens, a.H)) return ECHO_ESHAPE;
    }
    if (a.T == 0 || a.H == 0) return ECHO_OK;   // nothing to read or write: pointers may be NULL
    if (!backward && !a.r_out && !a.h) return ECHO_EINVAL;
    if (!a.x) return ECHO_EINVAL;
    if (!backward && a.h && a.h_dtype == ECHO_I8 && !a.h_scale) return ECHO_EINVAL;
    if (!aligned_elem(a.x, a.x_dtype) || (a.r && !aligned_elem(a.r, a.r_dtype)) ||
        (a.w_post && !aligned_elem(a.w_post, a.w_dtype)) || (a.w_pre && !aligned_elem(a.w_pre, a.w_dtype)) ||
        (a.gate && !aligned_elem(a.gate, a.w_dtype)))
        return ECHO_EALIGN;
    if (!backward && ((a.r_out && !aligned_elem(a.r_out, a.r_dtype)) || (a.h && !aligned_elem(a.h, a.h_dtype)) ||
                      (a.h && a.h_dtype == ECHO_I8 && !aligned_to(a.h_scale, 4))))
        return ECHO_EALIGN;
    return ECHO_OK;
}

echo::NormArgs norm_args(const echo_norm_args& a)
{
    echo::NormArgs n;
    std::memset(&n, 0, sizeof(n));
    n.x = a.x; n.r = a.r; n.w_post = a.w_post; n.w_pre = a.w_pre; n.gate = a.gate;
    n.r_out = a.r_out; n.h = a.h; n.h_scale = a.h_scale;
    n.T = a.T; n.ld_x = a.ld_x; n.ld_r = a.ld_r; n.ld_r_out = a.ld_r_out; n.ld_h = a.ld_h; n.ld_gate = a.ld_gate;
    n.gate_tokens = a.gate_tokens;
    n.H = (int)a.H;
    n.x_bf16 = a.x_dtype == ECHO_BF16; n.r_bf16 = a.r_dtype == ECHO_BF16; n.w_bf16 = a.w_dtype == ECHO_BF16;
    n.h_kind = a.h_dtype; n.post = a.post;
    n.eps = a.eps; n.rho = a.res_scale; n.beta = a.block_scale;
    return n;
}

}  // namespace

extern "C" {

int echo_quantize_tokens(const void* x, int64_t ldx, int x_dtype, int64_t T, int64_t K, int8_t* codes, int64_t ldq,
                         float* scales, void* stream)
{
    if (!float_dtype(x_dtype)) return ECHO_EUNSUP;
    if (bad_dim(T, kMaxRows) || bad_dim(K, echo::kI8MaxK)) return ECHO_ESHAPE;
    if (bad_ld(ldx, T, K) || bad_ld(ldq, T, K)) return ECHO_ESHAPE;
    if (T == 0) return ECHO_OK;
    if ((K && (!x || !codes)) || !scales) return ECHO_EINVAL;
    if (!aligned_elem(x, x_dtype) || !aligned_to(scales, 4)) return ECHO_EALIGN;
    echo::QuantTokArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = x; a.q = codes; a.scale = scales; a.ldx = ldx; a.ldq = ldq; a.T = T; a.K = (int)K;
    a.bf16 = x_dtype == ECHO_BF16;
    launch_quantize(a, (hipStream_t)stream);
    return check_launch();
}

int echo_gemm_int8(const int8_t* x, int64_t ldx, const float* sx, const int8_t* w, int64_t ldw, const float* sw,
                   const float* bias, int64_t M, int64_t N, int64_t K, void* y, int64_t ldy, int y_dtype, void* stream)
{
    const int rc = check_product(w, ldw, sw, bias, M, N, K, y, ldy, y_dtype);
    if (rc) return rc;
    if (bad_ld(ldx, M, K)) return ECHO_ESHAPE;
    if (M == 0 || N == 0) return ECHO_OK;
    if ((K && !x) || !sx) return ECHO_EINVAL;
    if (!aligned_to(sx, 4)) return ECHO_EALIGN;
    echo::GemmI8Args a = gemm_args(x, ldx, sx, w, ldw, sw, bias, M, N, K, y, ldy, y_dtype);
    launch_gemm_i8(a, (hipStream_t)stream);
    return check_launch();
}

size_t echo_linear_int8_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    if (bad_dim(M, kMaxRows) || bad_dim(N, kMaxRows) || bad_dim(K, echo::kI8MaxK)) return 0;
    return (size_t)(M * codes_ld(K) + 4 * M);
}

int echo_linear_int8(const void* x, int64_t ldx, int x_dtype, const int8_t* w, int64_t ldw, const float* sw,
                     const float* bias, int64_t M, int64_t N, int64_t K, void* y, int64_t ldy, int y_dtype,
                     void* workspace, size_t workspace_bytes, void* stream)
{
    if (!float_dtype(x_dtype)) return ECHO_EUNSUP;
    int rc = check_product(w, ldw, sw, bias, M, N, K, y, ldy, y_dtype);
    if (rc) return rc;
    if (bad_ld(ldx, M, K)) return ECHO_ESHAPE;
    if (M == 0 || N == 0) return ECHO_OK;
    if (K && !x) return ECHO_EINVAL;
    if (!aligned_elem(x, x_dtype)) return ECHO_EALIGN;
    if (!workspace || workspace_bytes < echo_linear_int8_workspace_bytes(M, N, K)) return ECHO_EINVAL;
    if (!aligned16(workspace)) return ECHO_EALIGN;
    const hipStream_t st = (hipStream_t)stream;
    const int64_t ldq = codes_ld(K);
    int8_t* q = (int8_t*)workspace;
    float* s = (float*)(q + M * ldq);
    echo::QuantTokArgs qa;
    std::memset(&qa, 0, sizeof(qa));
    qa.x = x; qa.q = q; qa.scale = s; qa.ldx = ldx; qa.ldq = ldq; qa.T = M; qa.K = (int)K;
    qa.bf16 = x_dtype == ECHO_BF16;
    launch_quantize(qa, st);
    if ((rc = check_launch())) return rc;
    echo::GemmI8Args a = gemm_args(q, ldq, s, w, ldw, sw, bias, M, N, K, y, ldy, y_dtype);
    launch_gemm_i8(a, st);
    return check_launch();
}

int echo_block_norm(const echo_norm_args* p, void* stream)
{
    const int rc = check_norm(p, false);
    if (rc || p->T == 0 || p->H == 0) return rc;
    const echo::NormArgs a = norm_args(*p);
    hipLaunchKernelGGL(echo::block_norm_any_kernel, dim3(grid_of(a.T)), dim3(echo::kBlock), 0, (hipStream_t)stream, a);
    return check_launch();
}

size_t echo_block_norm_backward_workspace_bytes(int64_t T, int64_t H)
{
    if (bad_dim(T, kMaxRows) || bad_dim(H, kMaxWidth)) return 0;
    return norm_stats_bytes(T) + (size_t)norm_chunks(T) * 2 * (size_t)H * 4;
}

int echo_block_norm_backward(const echo_norm_args* p, const echo_norm_grads* gp, void* stream)
{
    const int rc = check_norm(p, true);
    if (rc) return rc;
    if (!gp) return ECHO_EINVAL;
    const echo_norm_grads& g = *gp;
    const int64_t T = p->T, H = p->H;
    if (g.dh && !float_dtype(g.dh_dtype)) return ECHO_EUNSUP;
    if ((g.dh && bad_ld(g.ld_dh, T, H)) || (g.dr_out && bad_ld(g.ld_dr_out, T, H)) || (g.dx && bad_ld(g.ld_dx, T, H)) ||
        (g.dr && bad_ld(g.ld_dr, T, H)))
        return ECHO_ESHAPE;
    const int64_t rows = p->gate ? (T + p->gate_tokens - 1) / p->gate_tokens : 0;
    if (g.dgate && bad_ld(g.ld_dgate, rows, H)) return ECHO_ESHAPE;
    if ((g.dgate && !p->gate) || (g.dw_post && !p->post) || (g.dr && !p->r)) return ECHO_EINVAL;
    if (H == 0) return ECHO_OK;
    if (T > 0 && !g.dh && !g.dr_out) return ECHO_EINVAL;
    if ((g.dh && !aligned_elem(g.dh, g.dh_dtype)) || (g.dr_out && !aligned_elem(g.dr_out, p->r_dtype)) ||
        (g.dx && !aligned_elem(g.dx, p->x_dtype)) || (g.dr && !aligned_elem(g.dr, p->r_dtype)) ||
        !aligned_to(g.dw_post, 4) || !aligned_to(g.dw_pre, 4) || !aligned_to(g.dgate, 4))
        return ECHO_EALIGN;
    if (!g.workspace || g.workspace_bytes < echo_block_norm_backward_workspace_bytes(T, H)) return ECHO_EINVAL;
    if (!aligned16(g.workspace)) return ECHO_EALIGN;
    echo::NormBwdArgs b;
    std::memset(&b, 0, sizeof(b));
    b.f = norm_args(*p);
    b.dh = g.dh; b.dr_out = g.dr_out; b.dx = g.dx; b.dr = g.dr;
    b.dw_post = g.dw_post; b.dw_pre = g.dw_pre; b.dgate = g.dgate;
    b.ld_dh = g.ld_dh; b.ld_dr_out = g.ld_dr_out; b.ld_dx = g.ld_dx; b.ld_dr = g.ld_dr; b.ld_dgate = g.ld_dgate;
    b.dh_bf16 = g.dh_dtype == ECHO_BF16;
    b.stats = (float*)g.workspace;
    b.part = (float*)((uint8_t*)g.workspace + norm_stats_bytes(T));
    b.chunks = norm_chunks(T);
    const hipStream_t st = (hipStream_t)stream;
    const unsigned cols = (unsigned)((H + echo::kBlock - 1) / echo::kBlock);
    const dim3 block(echo::kBlock);
    int e;
    if (T > 0) {
        hipLaunchKernelGGL(echo::norm_bwd_stats_kernel, dim3(grid_of(T)), block, 0, st, b);
        if ((e = check_launch())) return e;
    }
    if (g.dw_post || g.dw_pre) {
        hipLaunchKernelGGL(echo::norm_bwd_weights_kernel, dim3(cols, (unsigned)b.chunks), block, 0, st, b);
        if ((e = check_launch())) return e;
        hipLaunchKernelGGL(echo::norm_bwd_weights_sum_kernel, dim3(cols), block, 0, st, b);
        if ((e = check_launch())) return e;
    }
    if (g.dgate && rows > 0) {
        hipLaunchKernelGGL(echo::norm_bwd_gate_kernel, dim3(cols, (unsigned)(rows < 32768 ? rows : 32768)), block, 0, st,
                           b, rows);
        if ((e = check_launch())) return e;
    }
    if (T > 0 && (g.dx || g.dr)) {
        hipLaunchKernelGGL(echo::norm_bwd_apply_kernel, dim3(grid_of(T)), block, 0, st, b);
        if ((e = check_launch())) return e;
    }
    return ECHO_OK;
}

}  // extern "C"
