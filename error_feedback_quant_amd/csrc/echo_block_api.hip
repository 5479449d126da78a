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
using echo::aligned_elem;
using echo::aligned_to;
using echo::bad_dim;
using echo::bad_ld;
using echo::check_launch;
using echo::float_dtype;
using echo::grid_fits;
using echo::grid_of;
using echo::kMaxRows;

template <int G, int C, bool BF16>
void quantize_go(const echo::QuantTokArgs& a, hipStream_t st)
{
    constexpr int kRows = echo::row_block<G>() / G;
    const dim3 grid(grid_of((a.T + kRows - 1) / kRows)), block(echo::row_block<G>());
    if (a.K % 8) hipLaunchKernelGGL((echo::quantize_tokens_kernel<G, C, BF16, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((echo::quantize_tokens_kernel<G, C, BF16, false>), grid, block, 0, st, a);
}

// The fewest threads that hold a token in two chunks each: a wave up to 1024
// elements (no barrier), then a block.
template <bool BF16>
void quantize_sized(const echo::QuantTokArgs& a, hipStream_t st)
{
    if (a.K <= 512) quantize_go<64, 1, BF16>(a, st);
    else if (a.K <= 1024) quantize_go<64, 2, BF16>(a, st);
    else if (a.K <= 4096) quantize_go<256, 2, BF16>(a, st);
    else if (a.K <= 16384) quantize_go<1024, 2, BF16>(a, st);
    else hipLaunchKernelGGL(echo::quantize_long_tokens_kernel, dim3(grid_of(a.T)), dim3(echo::kBlock), 0, st, a);
}

void launch_quantize(const echo::QuantTokArgs& a, hipStream_t st)
{
    if (a.bf16) quantize_sized<true>(a, st);
    else quantize_sized<false>(a, st);
}

// NR 0: no form of this tile for rows that start anywhere
template <int BM, int BN, int WM, int WN, int NS, int NR>
void gemm_stage_go(echo::GemmI8Args& a, bool direct, hipStream_t st)
{
    a.tiles_m = (uint32_t)((a.M + BM - 1) / BM);
    a.tiles_n = (uint32_t)((a.N + BN - 1) / BN);
    const dim3 grid(a.tiles_m * a.tiles_n), block(64 * WM * WN);
    if constexpr (NR > 0) {
        if (!direct) {
            hipLaunchKernelGGL((echo::gemm_i8_stage_kernel<BM, BN, WM, WN, 2, NR>), grid, block, 0, st, a);
            return;
        }
    }
    hipLaunchKernelGGL((echo::gemm_i8_stage_kernel<BM, BN, WM, WN, NS, 0>), grid, block, 0, st, a);
}

template <int MT, int XKIND, int FM, int C>
void gemm_few_go(const echo::GemmI8Args& a, const void* xf, hipStream_t st)
{
    echo::FewArgs f;
    f.g = a;
    f.xf = xf;
    f.pitch = echo::few_pitch(a.K);
    // every row of codes starts on a word
    const bool words = aligned_to(a.w, 4) && a.ldw % 4 == 0 && (XKIND || (aligned_to(a.x, 4) && a.ldx % 4 == 0));
    const size_t parts = (size_t)echo::kFewWaves * MT * 1024, codes = XKIND ? (size_t)a.M * f.pitch : 0;
    const size_t lds = parts > codes ? parts : codes;
    const dim3 grid((unsigned)((a.N + 15) / 16)), block(echo::kFewThreads);
    if (words) hipLaunchKernelGGL((echo::gemm_i8_few_kernel<MT, XKIND, FM, C, false>), grid, block, lds, st, f);
    else hipLaunchKernelGGL((echo::gemm_i8_few_kernel<MT, XKIND, FM, C, true>), grid, block, lds, st, f);
}

// Layers that one launch quantizes and multiplies, while the tokens fit the
// registers of gemm_i8_few_kernel: one token at N = K = 4096 takes 6.3 us, in
// two launches 8.5; four tokens 7.9 and 9.0.
constexpr int64_t kFusedTokens = 4, kFusedK = 2 * 8 * echo::kFewThreads;
bool linear_fused(int64_t M, int64_t N, int64_t K)
{
    return M <= kFusedTokens && K <= kFusedK && grid_fits((N + 15) / 16, echo::kFewThreads);
}

template <int XKIND>
void linear_fused_go(const echo::GemmI8Args& a, const void* x, hipStream_t st)
{
    const bool one = a.K <= kFusedK / 2;
    if (a.M == 1) one ? gemm_few_go<1, XKIND, 1, 1>(a, x, st) : gemm_few_go<1, XKIND, 1, 2>(a, x, st);
    else one ? gemm_few_go<1, XKIND, 4, 1>(a, x, st) : gemm_few_go<1, XKIND, 4, 2>(a, x, st);
}

// Tiles: one of the sizes below, by the estimated time of all rounds of tiles
// over the CUs.  `us` is a full chip's round of that tile at K = 4096 as
// measured, with direct loads and through registers.  A round also has a part
// that K does not change (256 x 256: 15.2 us at K = 256, 18.6 at 512, 24.4 at
// 1024, 61.9 at 4096), but the order of the tiles holds: of 17 sizes of 128 to
// 8192 tokens at K = 256 to 4096 the choice is the fastest tile for 15 and 4
// and 6 % behind for two; at 8192 x 8192 x 512 it took 87 us and 128 x 256 73.
// The largest tile reads the least per product and wins where it fills the
// chip (16384 x 4096 x 4096: 246 us, 276 with 128 x 256, 519 with 64 x 64);
// small calls want a tile for every CU, whose loads come at about 30 bytes a
// clock whatever the tile (100 x 4096 x 4096: 38 us with 256 x 256, 9.0 with
// 64 x 64, 7.9 with 64 x 32).  Through registers the largest tile spilled and
// gained nothing over the next one (4096 x 4096 x 3584).
struct TileCost {
    int bm, bn;
    float us[2];
};
constexpr TileCost kTiles[] = {{256, 256, {61.0f, 0.0f}},
                               {128, 256, {37.0f, 51.0f}},
                               {128, 128, {24.0f, 31.5f}},
                               {64, 128, {14.9f, 25.0f}},
                               {64, 64, {9.7f, 16.6f}},
                               {64, 32, {8.9f, 14.6f}}};
constexpr int64_t kCus = 256;

void launch_gemm_i8(echo::GemmI8Args& a, hipStream_t st)
{
    // Few tokens: the weight streams past them, without tiles, while the blocks
    // of 16 channels are about as many as the CUs.  Eight weights in turn, so
    // that they come from memory: 1 x 4096 x 4096 in 6.5 us (7.5 in 64 x 32
    // tiles), 8 tokens 7.3 (7.7), 16 8.1 (7.7), 32 9.9 (7.9); one weight that
    // stays in cache: 5.1 (7.1), 5.7 (7.2), 6.4 (7.1), 8.4 (7.5).  Each block
    // reads the tokens again, so with more channels only up to 8 of them (8 x
    // 8192 x 8192: 17.3 and 18.8, 16 tokens 19.0 and 19.1).
    if ((a.M <= 8 || (a.M <= 32 && a.N <= 16 * kCus)) && grid_fits((a.N + 15) / 16, echo::kFewThreads)) {
        if (a.M <= 16) gemm_few_go<1, 0, 1, 1>(a, nullptr, st);
        else gemm_few_go<2, 0, 1, 1>(a, nullptr, st);
        return;
    }
    const bool direct = aligned16(a.x) && aligned16(a.w) && a.ldx % 16 == 0 && a.ldw % 16 == 0;
    int best = -1;
    float least = 0.0f;
    for (int i = 0; i < (int)(sizeof(kTiles) / sizeof(kTiles[0])); ++i) {
        const int64_t tiles = ((a.M + kTiles[i].bm - 1) / kTiles[i].bm) * ((a.N + kTiles[i].bn - 1) / kTiles[i].bn);
        const float t = (float)((tiles + kCus - 1) / kCus) * kTiles[i].us[direct ? 0 : 1];
        if (t > 0.0f && grid_fits(tiles, 512) && (best < 0 || t < least)) {
            best = i;
            least = t;
        }
    }
    if (a.ldx >= echo::kI8StageLd || a.ldw >= echo::kI8StageLd) best = -1;
    switch (best) {
    case 0: return gemm_stage_go<256, 256, 2, 4, 2, 0>(a, direct, st);
    case 1: return gemm_stage_go<128, 256, 2, 4, 3, 2>(a, direct, st);
    case 2: return gemm_stage_go<128, 128, 2, 4, 4, 2>(a, direct, st);
    case 3: return gemm_stage_go<64, 128, 2, 2, 4, 2>(a, direct, st);
    case 4: return gemm_stage_go<64, 64, 2, 2, 4, 4>(a, direct, st);
    case 5: return gemm_stage_go<64, 32, 2, 1, 4, 2>(a, direct, st);
    default: break;
    }
    // rows too far apart for 32-bit offsets, or more tiles than a launch holds
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

// codes of the linear layer's tokens: rows of a multiple of 16, then the scales
int64_t codes_ld(int64_t K) { return (K + 15) / 16 * 16; }

echo::GemmI8Args gemm_args(const int8_t* x, int64_t ldx, const float* sx, const int8_t* w, int64_t ldw, const float* sw,
                           const float* bias, int64_t M, int64_t N, int64_t K, void* y, int64_t ldy, int y_dtype)
{
    echo::GemmI8Args a;
    std::memset(&a, 0, sizeof(a));
    a.x = x; a.w = w; a.sx = sx; a.sw = sw; a.bias = bias; a.y = y;
    a.M = M; a.N = N; a.ldy = ldy;
    a.ldx = M > 1 ? ldx : codes_ld(K);     // a single row's ld is not the caller's to set
    a.ldw = N > 1 ? ldw : codes_ld(K);
    a.K = (int)K; a.bf16 = y_dtype == ECHO_BF16;
    return a;
}

// ------------------------------------------------------------------ norms --

constexpr int64_t kMaxWidth = int64_t(1) << 30;
constexpr int64_t kBwdWidth = 8192;                 // rows whose backward pass fits a block's registers
size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

// f(G, C) for the threads and chunks that hold a row of H elements: a wave up
// to 1024 (no barrier), then whole blocks.  False: too long for registers.
template <typename F>
bool with_row_shape(int64_t H, F f)
{
    using std::integral_constant;
    if (H <= 512) f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    else if (H <= 1024) f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    else if (H <= 2048) f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
    else if (H <= 4096) f(integral_constant<int, 256>{}, integral_constant<int, 2>{});
    else if (H <= 8192) f(integral_constant<int, 512>{}, integral_constant<int, 2>{});
    else if (H <= 16384) f(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
    else return false;
    return true;
}

// The same for the backward pass, whose sums and weights take three times the
// registers: one chunk a thread.
template <typename F>
bool with_bwd_shape(int64_t H, F f)
{
    using std::integral_constant;
    if (H <= 512) f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    else if (H <= 1024) f(integral_constant<int, 128>{}, integral_constant<int, 1>{});
    else if (H <= 2048) f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
    else if (H <= 4096) f(integral_constant<int, 512>{}, integral_constant<int, 1>{});
    else if (H <= kBwdWidth) f(integral_constant<int, 1024>{}, integral_constant<int, 1>{});
    else return false;
    return true;
}

// How a backward pass is split, and where its parts lie in the workspace.
struct BwdPlan {
    int64_t blocks;          // of the row kernel; chunks of tokens for long rows
    int64_t per, groups;     // tokens of a group, groups that have any
    int group_shift;         // a block has 1 << group_shift groups
    size_t stats, part, gpart, total;
};
constexpr int64_t kBwdWaves = 8;
constexpr int64_t kMaxChunks = 256;

BwdPlan bwd_plan(int64_t T, int64_t H)
{
    BwdPlan p = {};
    if (T == 0) return p;                               // the sums' kernels then write zeros
    if (H > kBwdWidth) {
        p.blocks = T / 16 < 1 ? 1 : (T / 16 > kMaxChunks ? kMaxChunks : T / 16);
        while (!grid_fits(p.blocks, align256((size_t)H))) p.blocks /= 2;      // a column's thread in each chunk
        p.part = align256((size_t)(T * 16));
        p.total = p.part + (size_t)(p.blocks * 2 * H * 4);
        return p;
    }
    int threads = 0;
    with_bwd_shape(H, [&](auto g, auto) {
        threads = echo::row_block<decltype(g)::value>();
        for (p.group_shift = 0; (decltype(g)::value << p.group_shift) < threads; ++p.group_shift) {}
    });
    // two tokens a group at least, and 8 waves on a CU (more do not fit the
    // registers: 12 took 320 us at 131072 x 1024, 8 take 302) or one block
    int64_t most = kBwdWaves * 64 * kCus / threads;
    if (most < kCus) most = kCus;
    most <<= p.group_shift;
    const int64_t groups = (T + 1) / 2 < most ? (T + 1) / 2 : most;
    p.per = (T + groups - 1) / groups;
    p.groups = (T + p.per - 1) / p.per;
    p.blocks = (p.groups + (1 << p.group_shift) - 1) >> p.group_shift;
    p.gpart = align256((size_t)(p.blocks * 2 * H * 4));
    p.total = p.gpart + (size_t)((p.blocks << p.group_shift) * 2 * H * 4);
    return p;
}

// Groups of each gate row (1 row without a gate) where its tokens go round
// them, whole blocks to a row; 0 where that would leave a group with over an
// eighth more tokens than runs across the rows do.  131072 x 1024: 302 us,
// 334 in runs; with gate rows of 4096 tokens 324 and 336; 32768 x 4096 with
// gate rows of 2048 305 and 321.
uint32_t norm_spread(const BwdPlan& p, int64_t T, int64_t rows, int64_t gate_tokens)
{
    if (p.groups == 0) return 0;                        // no tokens, or a width without groups
    if (rows <= 1) return (uint32_t)(p.blocks << p.group_shift);
    const int64_t n = ((p.blocks << p.group_shift) / rows >> p.group_shift) << p.group_shift;
    return n > 0 && (gate_tokens + n - 1) / n * 8 <= p.per * 9 ? (uint32_t)n : 0;
}

// Tokens of a gate row that there are (gate_tokens may be any number from 1
// on), and the gate rows of T tokens.  The first bounds the second's sums:
// T + gate_tokens does not fit 64 bits for the largest gate_tokens.
int64_t gate_span(int64_t T, int64_t gate_tokens) { return gate_tokens < T ? gate_tokens : T; }
int64_t gate_row_count(int64_t T, int64_t gate_tokens)
{
    return T > 0 ? (T - 1) / gate_span(T, gate_tokens) + 1 : 0;
}

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
        if (bad_ld(a.ld_gate, gate_row_count(a.T, a.gate_tokens), a.H)) return ECHO_ESHAPE;
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
    n.gate_tokens = (uint32_t)gate_span(a.T, a.gate_tokens);
    n.H = (int)a.H;
    n.x_bf16 = a.x_dtype == ECHO_BF16; n.r_bf16 = a.r_dtype == ECHO_BF16; n.w_bf16 = a.w_dtype == ECHO_BF16;
    n.h_kind = a.h_dtype; n.post = a.post;
    n.eps = a.eps; n.rho = a.res_scale; n.beta = a.block_scale;
    return n;
}

// Blocks of a forward launch: those that the chip holds at once, each walking
// over its tokens with the weights in registers (2048 x 4096 in 23.5 us, 26.7
// with a block for each token), or, past kNormRounds rounds of them and
// without a gate, a block for each token, which keeps the chip on one stretch
// of memory (131072 x 1024: 182 us, 202 walking; with a gate to load for each
// token 196, 189 walking; rows of 8192, whose weights weigh more: 104 and 97).
constexpr int64_t kNormThreads = 1024 * kCus, kNormRounds = 8;

template <int G, int C, bool XB, bool RB>
void block_norm_go(const echo::NormArgs& a, hipStream_t st)
{
    constexpr int kThreads = echo::row_block<G>(), kRows = kThreads / G;
    int64_t blocks = (a.T + kRows - 1) / kRows;
    const int64_t held = kNormThreads / kThreads;
    if (blocks > held && (a.gate || G > 256 || blocks <= kNormRounds * held)) blocks = held;
    const dim3 grid(grid_of(blocks)), block(kThreads);
    if (a.H % 8) hipLaunchKernelGGL((echo::block_norm_kernel<G, C, XB, RB, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((echo::block_norm_kernel<G, C, XB, RB, false>), grid, block, 0, st, a);
}

void launch_block_norm(const echo::NormArgs& a, hipStream_t st)
{
    const bool held = with_row_shape(a.H, [&](auto g, auto c) {
        constexpr int G = decltype(g)::value, C = decltype(c)::value;
        if (a.x_bf16) a.r_bf16 ? block_norm_go<G, C, true, true>(a, st) : block_norm_go<G, C, true, false>(a, st);
        else a.r_bf16 ? block_norm_go<G, C, false, true>(a, st) : block_norm_go<G, C, false, false>(a, st);
    });
    if (!held)
        hipLaunchKernelGGL(echo::block_norm_any_kernel, dim3(grid_of(a.T)), dim3(echo::kBlock), 0, st, a);
}

template <int G, int C, bool XB, bool RB>
void block_norm_bwd_go(const echo::NormBwdArgs& b, hipStream_t st)
{
    const dim3 grid((unsigned)b.chunks), block(echo::row_block<G>());
    auto go = [&](auto hb, auto tail) {
        hipLaunchKernelGGL((echo::block_norm_bwd_kernel<G, C, XB, RB, decltype(hb)::value, decltype(tail)::value>), grid,
                           block, 0, st, b);
    };
    if (b.f.H % 8) b.dh_bf16 ? go(std::true_type{}, std::true_type{}) : go(std::false_type{}, std::true_type{});
    else b.dh_bf16 ? go(std::true_type{}, std::false_type{}) : go(std::false_type{}, std::false_type{});
}

int launch_block_norm_bwd(const echo::NormBwdArgs& b, const BwdPlan& plan, hipStream_t st)
{
    const echo::NormArgs& a = b.f;
    int e;
    if (a.T > 0) {
        with_bwd_shape(a.H, [&](auto g, auto c) {
            constexpr int G = decltype(g)::value, C = decltype(c)::value;
            if (a.x_bf16) a.r_bf16 ? block_norm_bwd_go<G, C, true, true>(b, st) : block_norm_bwd_go<G, C, true, false>(b, st);
            else a.r_bf16 ? block_norm_bwd_go<G, C, false, true>(b, st) : block_norm_bwd_go<G, C, false, false>(b, st);
        });
        if ((e = check_launch())) return e;
    }
    // gate rows that groups share; with a gate for each token there are none
    int64_t rows = b.dgate && (a.gate_tokens > 1 || b.spread) ? (plan.groups < b.gate_rows ? plan.groups : b.gate_rows) : 0;
    if (rows > 4096) rows = 4096;
    if (!b.dw_post && !b.dw_pre && !rows) return ECHO_OK;
    hipLaunchKernelGGL(echo::norm_bwd_sum_kernel, dim3((unsigned)((a.H + 63) / 64), (unsigned)(2 + rows)),
                       dim3(64 * echo::kSumWaves), 0, st, b, plan.group_shift);
    return check_launch();
}

// rows too long for registers: their statistics, then the sums by columns, then the rows' gradients
int launch_long_norm_bwd(const echo::NormBwdArgs& b, hipStream_t st)
{
    const echo::NormArgs& a = b.f;
    const unsigned cols = (unsigned)((a.H + echo::kBlock - 1) / echo::kBlock);
    const dim3 block(echo::kBlock);
    int e;
    if (a.T > 0) {
        hipLaunchKernelGGL(echo::norm_bwd_stats_kernel, dim3(grid_of(a.T)), block, 0, st, b);
        if ((e = check_launch())) return e;
    }
    if (b.dw_post || b.dw_pre) {
        if (b.chunks) {
            hipLaunchKernelGGL(echo::norm_bwd_weights_kernel, dim3(cols, (unsigned)b.chunks), block, 0, st, b);
            if ((e = check_launch())) return e;
        }
        hipLaunchKernelGGL(echo::norm_bwd_weights_sum_kernel, dim3(cols), block, 0, st, b);
        if ((e = check_launch())) return e;
    }
    if (b.dgate && b.gate_rows > 0) {
        uint32_t gy = b.gate_rows < 32768 ? b.gate_rows : 32768;              // the kernel strides over the rest
        while (!grid_fits((int64_t)cols * gy, echo::kBlock)) gy /= 2;
        hipLaunchKernelGGL(echo::norm_bwd_gate_kernel, dim3(cols, gy), block, 0, st, b);
        if ((e = check_launch())) return e;
    }
    if (a.T > 0 && (b.dx || b.dr)) {
        hipLaunchKernelGGL(echo::norm_bwd_apply_kernel, dim3(grid_of(a.T)), block, 0, st, b);
        if ((e = check_launch())) return e;
    }
    return ECHO_OK;
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
    return linear_fused(M, N, K) ? 0 : (size_t)(M * codes_ld(K) + 4 * M);
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
    const size_t need = echo_linear_int8_workspace_bytes(M, N, K);
    if (need && (!workspace || workspace_bytes < need)) return ECHO_EINVAL;
    if (!aligned16(workspace)) return ECHO_EALIGN;
    const hipStream_t st = (hipStream_t)stream;
    if (linear_fused(M, N, K)) {
        const echo::GemmI8Args a = gemm_args(nullptr, ldx, nullptr, w, ldw, sw, bias, M, N, K, y, ldy, y_dtype);
        if (x_dtype == ECHO_BF16) linear_fused_go<1>(a, x, st);
        else linear_fused_go<2>(a, x, st);
        return check_launch();
    }
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
    if (rc || p->T == 0) return rc;
    if (p->H == 0) {        // tokens of no elements have the scales that quantizing them gives
        if (p->h_dtype != ECHO_I8 || !p->h_scale) return ECHO_OK;
        return echo_quantize_tokens(nullptr, 0, ECHO_F32, p->T, 0, nullptr, 0, p->h_scale, stream);
    }
    const echo::NormArgs a = norm_args(*p);
    launch_block_norm(a, (hipStream_t)stream);
    return check_launch();
}

size_t echo_block_norm_backward_workspace_bytes(int64_t T, int64_t H)
{
    if (bad_dim(T, kMaxRows) || bad_dim(H, kMaxWidth)) return 0;
    return bwd_plan(T, H).total;
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
    const int64_t rows = p->gate ? gate_row_count(T, p->gate_tokens) : 0;
    if (g.dgate && bad_ld(g.ld_dgate, rows, H)) return ECHO_ESHAPE;
    if ((g.dgate && !p->gate) || (g.dw_post && !p->post) || (g.dr && !p->r)) return ECHO_EINVAL;
    if (H == 0) return ECHO_OK;
    if (T > 0 && !g.dh && !g.dr_out) return ECHO_EINVAL;
    if ((g.dh && !aligned_elem(g.dh, g.dh_dtype)) || (g.dr_out && !aligned_elem(g.dr_out, p->r_dtype)) ||
        (g.dx && !aligned_elem(g.dx, p->x_dtype)) || (g.dr && !aligned_elem(g.dr, p->r_dtype)) ||
        !aligned_to(g.dw_post, 4) || !aligned_to(g.dw_pre, 4) || !aligned_to(g.dgate, 4))
        return ECHO_EALIGN;
    const size_t need = echo_block_norm_backward_workspace_bytes(T, H);
    if (need && (!g.workspace || g.workspace_bytes < need)) return ECHO_EINVAL;
    if (!aligned16(g.workspace)) return ECHO_EALIGN;
    echo::NormBwdArgs b;
    std::memset(&b, 0, sizeof(b));
    b.f = norm_args(*p);
    b.dh = g.dh; b.dr_out = g.dr_out; b.dx = g.dx; b.dr = g.dr;
    b.dw_post = g.dw_post; b.dw_pre = g.dw_pre; b.dgate = g.dgate;
    b.ld_dh = g.ld_dh; b.ld_dr_out = g.ld_dr_out; b.ld_dx = g.ld_dx; b.ld_dr = g.ld_dr; b.ld_dgate = g.ld_dgate;
    b.dh_bf16 = g.dh_dtype == ECHO_BF16;
    const BwdPlan plan = bwd_plan(T, H);
    uint8_t* ws = (uint8_t*)g.workspace;
    b.stats = (float*)(ws + plan.stats);
    b.part = (float*)(ws + plan.part);
    b.gpart = (float*)(ws + plan.gpart);
    b.chunks = T > 0 ? (int)plan.blocks : 0;
    b.per = (uint32_t)plan.per;
    b.groups = (uint32_t)plan.groups;
    b.gate_rows = (uint32_t)rows;
    b.spread = norm_spread(plan, T, rows, b.f.gate_tokens);
    if (b.spread) b.chunks = (int)((rows > 1 ? rows : 1) * (b.spread >> plan.group_shift));
    const hipStream_t st = (hipStream_t)stream;
    return H > kBwdWidth ? launch_long_norm_bwd(b, st) : launch_block_norm_bwd(b, plan, st);
}

}  // extern "C"
