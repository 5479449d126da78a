// echo_int4_api.hip — host side of the linear layer with 4-bit weights:
// argument checks and launches; semantics, layouts and error behaviour are
// specified in include/echo.h.
#include <hip/hip_runtime.h>

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

bool known_group(int group) { return group == 32 || group == 64 || group == 128 || group == 256; }
int64_t groups_of(int64_t K, int group) { return (K + group - 1) / group; }

template <int L>
void quantize_go(const echo::QuantGroupArgs& a, bool bf16, hipStream_t st)
{
    const int64_t per = int64_t(1) << a.shift, rows = echo::kBlock >> a.shift;
    const int64_t chunks = ((int64_t)a.K + 8 * per - 1) / (8 * per);       // of a row, for its threads
    const dim3 grid(grid_of((a.T + rows - 1) / rows), (unsigned)(chunks < 1024 ? chunks : 1024)), block(echo::kBlock);
    if (bf16) hipLaunchKernelGGL((echo::quantize_groups_kernel<L, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((echo::quantize_groups_kernel<L, false>), grid, block, 0, st, a);
}

constexpr int64_t kMostTiles = (int64_t(1) << 23) - 1;  // of 16 channels by 32 tokens: a launch's threads stay in 32 bits

template <int GROUP, int MT, int NT, int DEPTH, bool BF16>
void linear_go(const echo::Int4Args& a, hipStream_t st)
{
    const dim3 grid((unsigned)((a.N + 16 * NT - 1) / (16 * NT)), (unsigned)((a.M + 16 * MT - 1) / (16 * MT)));
    hipLaunchKernelGGL((echo::linear_int4_kernel<GROUP, MT, NT, DEPTH, BF16>), grid, dim3(echo::kInt4Threads), 0, st, a);
}
#ifndef N4
#define N4 2
#endif
#ifndef D1
#define D1 4
#endif
#ifndef D2
#define D2 2
#endif

// fp32 tokens are three operands each, so a block takes half as many
template <int GROUP>
void linear_sized(const echo::Int4Args& a, bool x_bf16, hipStream_t st)
{
    constexpr int kUnits = GROUP == 256 ? 1 : 2;             // of 256 elements
    if (x_bf16) {
        if (a.M <= 16) linear_go<GROUP, 1, 1, kUnits * D1 / 2, true>(a, st);
        else if (a.M <= 32) linear_go<GROUP, 2, 1, kUnits * D2 / 2, true>(a, st);
        else linear_go<GROUP, 4, N4, 1, true>(a, st);
    } else {
        if (a.M <= 16) linear_go<GROUP, 1, 1, kUnits, false>(a, st);
        else linear_go<GROUP, 2, 1, 1, false>(a, st);
    }
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

size_t echo_linear_int4_workspace_bytes(int64_t, int64_t, int64_t, int) { return 0; }

int echo_linear_int4(const void* x, int64_t ldx, int x_dtype, const uint8_t* w, int64_t ldw, const echo_qparam* params,
                     int64_t ldp, int group, const float* bias, int64_t M, int64_t N, int64_t K, void* y, int64_t ldy,
                     int y_dtype, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!float_dtype(x_dtype) || !float_dtype(y_dtype) || !known_group(group)) return ECHO_EUNSUP;
    if (bad_dim(M, kMaxRows) || bad_dim(N, kMaxRows) || bad_dim(K, kMaxK)) return ECHO_ESHAPE;
    if (bad_ld(ldx, M, K) || bad_ld(ldw, N, (K + 1) / 2) || bad_ld(ldp, N, groups_of(K, group)) || bad_ld(ldy, M, N))
        return ECHO_ESHAPE;
    if ((M + 31) / 32 * ((N + 15) / 16) > kMostTiles || M > 32 * 65535) return ECHO_ESHAPE;
    if (M == 0 || N == 0) return ECHO_OK;
    if ((K && (!x || !w || !params)) || !y) return ECHO_EINVAL;
    if (!aligned_elem(x, x_dtype) || !aligned_to(params, 4) || !aligned_to(bias, 4) || !aligned_elem(y, y_dtype))
        return ECHO_EALIGN;
    const size_t need = echo_linear_int4_workspace_bytes(M, N, K, group);
    if (need && (!workspace || workspace_bytes < need)) return ECHO_EINVAL;
    if (!aligned16(workspace)) return ECHO_EALIGN;
    echo::Int4Args a;
    std::memset(&a, 0, sizeof(a));
    a.x = x; a.w = w; a.p = (const uint32_t*)params; a.bias = bias; a.y = y;
    a.M = M; a.N = N; a.ldx = ldx; a.ldw = ldw; a.ldp = ldp; a.ldy = ldy; a.K = (int)K; a.bf16 = y_dtype == ECHO_BF16;
    const bool xb = x_dtype == ECHO_BF16;
    const hipStream_t st = (hipStream_t)stream;
    switch (group) {
    case 32: linear_sized<32>(a, xb, st); break;
    case 64: linear_sized<64>(a, xb, st); break;
    case 128: linear_sized<128>(a, xb, st); break;
    default: linear_sized<256>(a, xb, st); break;
    }
    return check_launch();
}

}  // extern "C"
