// echo_int4_api.hip — host side of the linear layer with 4-bit weights:
// argument checks and launches; semantics, layouts and error behaviour are
// specified in include/echo.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "echo.h"
#include "echo_host.hpp"
#include "echo_int4.hpp"

namespace {

using echo::aligned16;
using echo::aligned_elem;
using echo::aligned_to;
using echo::bad_dim;
using echo::bad_ld;
using echo::check_launch;
using echo::float_dtype;
using echo::grid_of;
using echo::kMaxRows;

constexpr int64_t kMaxK = int64_t(1) << 30;
constexpr int64_t kMostX = int64_t(1) << 36;            // elements of x: its fragments' threads stay in 32 bits

bool known_group(int group) { return group == 32 || group == 64 || group == 128 || group == 256; }
int64_t groups_of(int64_t K, int group) { return (K + group - 1) / group; }

template <int L>
void quantize_go(const echo::QuantGroupArgs& a, bool bf16, hipStream_t st)
{
    const int64_t per = int64_t(1) << a.shift, rows = echo::kBlock >> a.shift;
    const int64_t chunks = ((int64_t)a.K + 8 * per - 1) / (8 * per);       // of a row, for its threads
    const int64_t x = grid_of((a.T + rows - 1) / rows), y = std::min({chunks, int64_t(1024), (int64_t(1) << 23) / x});
    const dim3 grid((unsigned)x, (unsigned)y), block(echo::kBlock);      // the kernel strides over the rest
    if (bf16) hipLaunchKernelGGL((echo::quantize_groups_kernel<L, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((echo::quantize_groups_kernel<L, false>), grid, block, 0, st, a);
}

constexpr int64_t kMostTiles = (int64_t(1) << 23) - 1;  // of 16 channels by 32 tokens: a launch's threads stay in 32 bits

// Up to 16 tokens one launch reads x as it is; more are laid out first, for
// blocks of 64 tokens (32 in fp32) by 32 channels, or 16 where those are too
// few for the CUs.  Up to 32 bf16 tokens of a small layer, in rows that start
// at 8 bytes, still go faster as they are (us for 27 tokens, as they are and
// laid out: 2048 x 2048 8.8, 11.3, 4096 x 4096 10.9, 11.5, 8192 x 8192 31, 21;
// 1001 x 3583 in rows at odd words 22.8, 11.6).
int64_t tokens_of_block(bool x_bf16) { return x_bf16 ? 64 : 32; }
bool as_it_is(const void* x, int64_t ldx, int64_t M, int64_t N, int64_t K, bool x_bf16)
{
    if (M <= 16 || K == 0) return true;
    return x_bf16 && M <= 32 && N * K < (int64_t(1) << 25) && aligned_to(x, 8) && ldx % 4 == 0;
}

struct Int4Layout {
    int64_t units, tiles;   // of K, of 16 tokens (whole blocks)
    size_t xs, total;       // of the workspace
};
Int4Layout int4_layout(int64_t M, int64_t K, int group, bool x_bf16)
{
    Int4Layout l = {};
    if (M <= 16 || K == 0) return l;
    const int64_t unit = group < 128 ? 128 : group, most = M <= 32 ? 32 : tokens_of_block(x_bf16);
    l.units = (K + unit - 1) / unit;
    l.tiles = (M + most - 1) / most * (most / 16);
    l.xs = (size_t)(l.units * l.tiles * (unit / 32) * (x_bf16 ? 1 : 3) * 1024);
    l.total = l.xs + (size_t)(l.units * l.tiles * (unit / group) * 64);
    return l;
}

template <int GROUP, int MT, int DEPTH, bool BF16>
void linear_go(const echo::Int4Args& a, hipStream_t st)
{
    const dim3 grid((unsigned)((a.N + 15) / 16), (unsigned)((a.M + 16 * MT - 1) / (16 * MT)));
    hipLaunchKernelGGL((echo::linear_int4_kernel<GROUP, MT, DEPTH, BF16>), grid, dim3(echo::kInt4Threads), 0, st, a);
}
template <int GROUP, int MT, int P>
void linear_tile_go(const echo::Int4Tiles& b, hipStream_t st)
{
    const unsigned rows = (unsigned)(b.tiles / MT);
    const dim3 wide((unsigned)((b.a.N + 31) / 32), rows), narrow((unsigned)((b.a.N + 15) / 16), rows), block(echo::kInt4Threads);
    if ((int64_t)wide.x * rows >= 256) hipLaunchKernelGGL((echo::linear_int4_tile_kernel<GROUP, MT, 2, P>), wide, block, 0, st, b);
    else hipLaunchKernelGGL((echo::linear_int4_tile_kernel<GROUP, MT, 1, P>), narrow, block, 0, st, b);
}

template <int GROUP>
int linear_sized(const echo::Int4Args& a, bool x_bf16, void* workspace, const Int4Layout& l, hipStream_t st)
{
    if (as_it_is(a.x, a.ldx, a.M, a.N, a.K, x_bf16)) {
        constexpr int kUnits = GROUP == 256 ? 2 : 4;         // fp32 tokens are three operands each
        if (!x_bf16 && a.M <= 16) linear_go<GROUP, 1, kUnits / 2, false>(a, st);
        else if (a.M <= 16) linear_go<GROUP, 1, kUnits, true>(a, st);
        else linear_go<GROUP, 2, kUnits / 2, true>(a, st);   // more than 32, or of fp32, where K is 0: nothing is read
        return check_launch();
    }
    echo::Int4Tiles b;
    std::memset(&b, 0, sizeof(b));
    b.a = a;
    b.x = (echo::bf16x8*)workspace;
    b.xs = (echo::f32x4*)((uint8_t*)workspace + l.xs);
    b.units = (int)l.units;
    b.tiles = (int)l.tiles;
    const dim3 grid((unsigned)((l.units * l.tiles + 3) / 4)), block(echo::kBlock);
    if (x_bf16) hipLaunchKernelGGL((echo::arrange_int4_kernel<GROUP, true>), grid, block, 0, st, b);
    else hipLaunchKernelGGL((echo::arrange_int4_kernel<GROUP, false>), grid, block, 0, st, b);
    const int e = check_launch();
    if (e) return e;
    if (x_bf16) a.M <= 32 ? linear_tile_go<GROUP, 2, 1>(b, st) : linear_tile_go<GROUP, 4, 1>(b, st);
    else linear_tile_go<GROUP, 2, 3>(b, st);
    return check_launch();
}

}  // namespace

extern "C" {

int echo_quantize_groups(const void* x, int64_t ldx, int x_dtype, int64_t T, int64_t K, int group, uint8_t* codes,
                         int64_t ldq, echo_qparam* params, int64_t ldp, void* stream)
{
    if (!float_dtype(x_dtype) || !known_group(group)) return ECHO_EUNSUP;
    if (bad_dim(T, kMaxRows) || bad_dim(K, kMaxK)) return ECHO_ESHAPE;
    if (bad_ld(ldx, T, K) || bad_ld(ldq, T, (K + 1) / 2) || bad_ld(ldp, T, groups_of(K, group))) return ECHO_ESHAPE;
    if (T == 0 || K == 0) return ECHO_OK;
    if (!x || !codes || !params) return ECHO_EINVAL;
    if (!aligned_elem(x, x_dtype) || !aligned_to(params, 4)) return ECHO_EALIGN;
    echo::QuantGroupArgs a;
    std::memset(&a, 0, sizeof(a));
    a.x = x; a.q = codes; a.p = (uint32_t*)params; a.ldx = ldx; a.ldq = ldq; a.ldp = ldp; a.T = T; a.K = (int)K;
    a.shift = 2;
    while ((8 << a.shift) < group) ++a.shift;
    while (a.shift < 8 && (int64_t(8) << a.shift) < K) ++a.shift;
    const bool bf16 = x_dtype == ECHO_BF16;
    const hipStream_t st = (hipStream_t)stream;
    switch (group) {
    case 32: quantize_go<4>(a, bf16, st); break;
    case 64: quantize_go<8>(a, bf16, st); break;
    case 128: quantize_go<16>(a, bf16, st); break;
    default: quantize_go<32>(a, bf16, st); break;
    }
    return check_launch();
}

size_t echo_linear_int4_workspace_bytes(int64_t M, int64_t N, int64_t K, int group)
{
    if (bad_dim(M, kMaxRows) || bad_dim(N, kMaxRows) || bad_dim(K, kMaxK) || !known_group(group) || N == 0) return 0;
    if (M > 32 * 65535 || M * K > kMostX) return 0;
    // x's type is not among the arguments: room for the larger
    return std::max(int4_layout(M, K, group, true).total, int4_layout(M, K, group, false).total);
}

int echo_linear_int4(const void* x, int64_t ldx, int x_dtype, const uint8_t* w, int64_t ldw, const echo_qparam* params,
                     int64_t ldp, int group, const float* bias, int64_t M, int64_t N, int64_t K, void* y, int64_t ldy,
                     int y_dtype, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!float_dtype(x_dtype) || !float_dtype(y_dtype) || !known_group(group)) return ECHO_EUNSUP;
    if (bad_dim(M, kMaxRows) || bad_dim(N, kMaxRows) || bad_dim(K, kMaxK)) return ECHO_ESHAPE;
    if (bad_ld(ldx, M, K) || bad_ld(ldw, N, (K + 1) / 2) || bad_ld(ldp, N, groups_of(K, group)) || bad_ld(ldy, M, N))
        return ECHO_ESHAPE;
    if ((M + 31) / 32 * ((N + 15) / 16) > kMostTiles || M > 32 * 65535 || M * K > kMostX) return ECHO_ESHAPE;
    if (M == 0 || N == 0) return ECHO_OK;
    if ((K && (!x || !w || !params)) || !y) return ECHO_EINVAL;
    if (!aligned_elem(x, x_dtype) || !aligned_to(params, 4) || !aligned_to(bias, 4) || !aligned_elem(y, y_dtype))
        return ECHO_EALIGN;
    const bool xb = x_dtype == ECHO_BF16;
    const Int4Layout l = int4_layout(M, K, group, xb);
    const size_t need = echo_linear_int4_workspace_bytes(M, N, K, group);
    if (need && (!workspace || workspace_bytes < need)) return ECHO_EINVAL;
    if (!aligned16(workspace)) return ECHO_EALIGN;
    echo::Int4Args a;
    std::memset(&a, 0, sizeof(a));
    a.x = x; a.w = w; a.p = (const uint32_t*)params; a.bias = bias; a.y = y;
    a.M = M; a.N = N; a.ldx = ldx; a.ldw = ldw; a.ldp = ldp; a.ldy = ldy; a.K = (int)K; a.bf16 = y_dtype == ECHO_BF16;
    const hipStream_t st = (hipStream_t)stream;
    switch (group) {
    case 32: return linear_sized<32>(a, xb, workspace, l, st);
    case 64: return linear_sized<64>(a, xb, workspace, l, st);
    case 128: return linear_sized<128>(a, xb, workspace, l, st);
    default: return linear_sized<256>(a, xb, workspace, l, st);
    }
}

}  // extern "C"
