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

#include <type_traits>

#include "echo_kernels.hpp"
#include "echo_rows.hpp"
#include "echo_stage.hpp"

namespace echo {

constexpr int kI8MaxK = (1 << 17) - 1;       // 2^14 * K stays below 2^31

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

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

// A token held in registers: G threads with C chunks of 8 elements each, one
// pass over memory.  Bound by memory: 16384 x 4096 bf16 (201 MB) in 36 us, 5.6
// TB/s, with four inputs in turn (64, 128 or 512 threads a token: 37.7, 36.4,
// 38.3), in 43 behind a product that has had the caches, in 30 with its input
// still there; 27 x 3584 in 2.7.
template <int G, int C, bool BF16, bool TAIL>
__global__ __launch_bounds__(row_block<G>()) void quantize_tokens_kernel(const QuantTokArgs a)
{
    __shared__ float red[G > 64 ? 2 * G / 64 : 1];
    constexpr int kRows = row_block<G>() / G;
    const int g = threadIdx.x % G;
    int turn = 0;
    for (int64_t t = (int64_t)blockIdx.x * kRows + threadIdx.x / G; t < a.T; t += (int64_t)gridDim.x * kRows) {
        Raw8<BF16> x[C];
#pragma unroll
        for (int j = 0; j < C; ++j) x[j] = ld_raw8<BF16, TAIL>(a.x, t * a.ldx, 8 * (g + G * j), a.K);
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < C; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) m = max(m, abs_bits(raw_get(x[j], e)));
        const TokenScale s = token_scale(row_max_u32<G>(m, red, turn++));
#pragma unroll
        for (int j = 0; j < C; ++j) {
            int q[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] = token_code(raw_get(x[j], e), s.inv);
            st_codes8<TAIL>(a.q, t * a.ldq, 8 * (g + G * j), a.K, q);
        }
        if (g == 0) a.scale[t] = s.scale;
    }
}

// Tokens longer than a block's registers: one block per token, two passes by
// single elements (2048 x 20000 in bf16, 123 MB, takes 62 us).
__global__ __launch_bounds__(kBlock) void quantize_long_tokens_kernel(const QuantTokArgs a)
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
// read: the last row of an operand may end where its allocation ends.  Where
// the row ends inside them, the last 16 bytes of the row are read and shifted
// down (byte by byte they took 8 us of a 26 us call).  Any alignment: gfx950
// loads 16 unaligned bytes in one access.
__device__ __forceinline__ i32x4 ld_codes16(const int8_t* row, int k, int K)
{
    i32x4 v = {0, 0, 0, 0};
    if (k + 16 <= K) {
        __builtin_memcpy(&v, row + k, 16);
    } else if (k < K && K >= 16) {
        uint64_t w[2];
        __builtin_memcpy(w, row + K - 16, 16);
        const uint32_t bits = 8u * (uint32_t)(k + 16 - K);   // 8 .. 120
        const uint64_t lo = bits >= 64 ? w[1] >> (bits - 64) : (w[0] >> bits) | (w[1] << (64 - bits));
        const uint64_t hi = bits >= 64 ? 0 : w[1] >> bits;
        v = i32x4{(int)lo, (int)(lo >> 32), (int)hi, (int)(hi >> 32)};
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
// steps of 64 bytes through registers into LDS, blocks striding over the
// tiles and 64-bit offsets throughout.  It serves what the kernels below do
// not: rows at 4 MB and more from one another, and more tiles than one launch
// holds (4096 x 4096 x 3584 takes it 172 us, them 55).
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

// ---------------------------------------------------------------- tiles --
//
// A BM x BN output tile per block of WM x WN waves, K in stages of 128 bytes.
// The weight is the first MFMA operand, so a lane's accumulators run along n
// and leave as whole vectors.
//
// NR = 0: rows start at multiples of 16 bytes.  Stages are filled by 16-byte
// buffer loads straight into LDS, NS of them in turn: while a stage is
// multiplied the next NS - 1 are on their way.  NR > 0: rows start anywhere;
// the next stages wait in NR sets of registers, shifted into place when they
// move to one of two stages in LDS.
//
// Order of one stage (four steps of 32 bytes, fragments in two register
// sets): the last step's fragments are in registers before the stage ends, so
// the barrier that releases the stage stands before that step's MFMAs, and
// the first fragments of the next stage are read under them; a barrier at the
// stage's end would leave the matrix cores idle for an LDS round trip.
//
// Measured (direct loads): 4096 x 4096 x 3584 in 54 us (2.21 POP/s; 58 after a
// while of full load), 16384 x 4096 x 4096 in 246 to 267 by the clock it gets,
// 255 behind its quantization (2.16 POP/s).  With 256 x 256 tiles the matrix
// cores are busy for 62 % of a tile's cycles; a full chip runs at about 1.8 GHz
// (half of it at 2.4: 63 us for 256 tiles of K = 4096, 46 for 128), so beyond
// that power bounds it: the 4-wave form of the tile, with a third less LDS
// traffic but one wave on each SIMD, took 62 us.  Small tiles are bound by
// their loads, which come at about 30 bytes a clock and CU whatever the tile;
// splitting K over two halves of a block, or reading a whole stage's
// fragments at once, made them no faster.  Rows at odd places need a fifth
// word for each 16 bytes and more lines: 91 us at 4096 x 4096 x 3584.

constexpr int kI8BK = 128;                   // bytes of K per stage
constexpr int64_t kI8StageLd = int64_t(1) << 22;   // row distances below this keep a panel's offsets in 31 bits
constexpr uint32_t kXcds = 8;

// Output tile of block b: each XCD (b mod 8) takes a contiguous run of a
// grouped order (8 tile rows, column by column), a compact patch whose
// panels stay in its L2.
__device__ __forceinline__ void xcd_tile_of(uint32_t b, uint32_t tiles_m, uint32_t tiles_n, uint32_t& tm, uint32_t& tn)
{
    const uint32_t T = tiles_m * tiles_n;
    const uint32_t x = b % kXcds, each = T / kXcds, more = T % kXcds;
    const uint32_t t = x * each + min(x, more) + b / kXcds;
    const uint32_t group = t / (8u * tiles_n);
    const uint32_t rows = min(tiles_m - 8u * group, 8u);
    const uint32_t in = t - group * 8u * tiles_n;
    tm = 8u * group + in % rows;
    tn = in / rows;
}

// s_waitcnt operand: at most `left` vector-memory operations outstanding
constexpr int waitcnt_vm(int left) { return 0x0F70 | (left & 15) | ((left >> 4) << 14); }

// A barrier of the block that leaves `LEFT` vector-memory operations of each
// wave on their way (and no LDS operation).  __syncthreads() would wait for
// all of them, and so for the stages that are meant to be under way.
template <int LEFT>
__device__ __forceinline__ void stage_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");   // for the compiler: no access moves across
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(LEFT) & 0xF0FF);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
}

// 16 bytes of each lane from its offset, behind k0, to 16 bytes a lane of LDS
__device__ __forceinline__ void stage_load16(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t k0, uint8_t* lds)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, off, k0, 0, 0);
}

template <int BM, int BN, int WM, int WN, int NS, int NR>
__global__ __launch_bounds__(64 * WM * WN) __attribute__((amdgpu_waves_per_eu(WM * WN / 4, WM * WN / 4)))
void gemm_i8_stage_kernel(const GemmI8Args a)
{
    constexpr bool DIRECT = NR == 0;
    static_assert(DIRECT || NS == 2, "stages wait in registers, not in LDS");
    constexpr int NW = WM * WN, NT = 64 * NW;
    constexpr int TM = BM / WM / 32, TN = BN / WN / 32;      // 32 x 32 fragments of a wave
    constexpr int kStage = (BM + BN) * kI8BK;
    constexpr int LM = BM / (8 * NW), LN = BN / (8 * NW);    // loads of a thread per stage
    constexpr int CW = BN / WN;                              // columns of a wave
    constexpr int kPitch = CW + 4;                           // ints; shifts rows by four banks in the epilogue
    static_assert(NW * 32 * kPitch * 4 <= NS * kStage, "the epilogue fits the stages");
    __shared__ __align__(16) uint8_t smem[NS * kStage];

    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t wm = wave / WN, wn = wave % WN;
    uint32_t tm, tn;
    xcd_tile_of(blockIdx.x, a.tiles_m, a.tiles_n, tm, tn);
    const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
    const int rows_m = (int)min((int64_t)BM, a.M - m0), rows_n = (int)min((int64_t)BN, a.N - n0);
    const int8_t* px = a.x + m0 * a.ldx;
    const int8_t* pw = a.w + n0 * a.ldw;
    const uint32_t ldx = (uint32_t)a.ldx, ldw = (uint32_t)a.ldw;
    const __amdgpu_buffer_rsrc_t rx =
        __builtin_amdgcn_make_buffer_rsrc((void*)px, (short)0, (int)((rows_m - 1) * ldx + a.K), 0x00020000);
    const __amdgpu_buffer_rsrc_t rw =
        __builtin_amdgcn_make_buffer_rsrc((void*)pw, (short)0, (int)((rows_n - 1) * ldw + a.K), 0x00020000);

    // a wave's load moves 8 rows; lane i lands 16 i bytes behind the wave's
    // base, so it fetches the chunk that belongs there
    const uint32_t lrow = wave * 8 + (lane >> 3);
    const uint32_t lchunk = (lane & 7u) ^ i8_key(lrow);
    uint32_t off[LM + LN];                                   // of a stage's loads: LM of x, then LN of w
#pragma unroll
    for (int i = 0; i < LM + LN; ++i) {
        const uint32_t r = lrow + 8 * NW * (i < LM ? i : i - LM);
        off[i] = i < LM ? stage_offset(r, (uint32_t)rows_m, ldx, lchunk) : stage_offset(r, (uint32_t)rows_n, ldw, lchunk);
    }
    auto issue1 = [&](int i, uint32_t buf, uint32_t k0) {
        uint8_t* to = smem + buf * kStage + (i < LM ? 0 : BM * kI8BK);
        const int j = i < LM ? i : i - LM;
        stage_load16(i < LM ? rx : rw, off[i], k0, to + (8 * NW * j + wave * 8) * kI8BK);
    };
    auto issue = [&](uint32_t buf, uint32_t k0) {
#pragma unroll
        for (int i = 0; i < LM + LN; ++i) issue1(i, buf, k0);
    };
    // The same through NR sets of registers, for rows that start anywhere.  The
    // words that hold the 16 bytes are loaded and shifted together: 16-byte
    // loads at odd addresses ran at under half the rate.
    constexpr int kSets = DIRECT ? 1 : NR, kHeld = DIRECT ? 1 : LM + LN;
    u32x4 held[kSets][kHeld];
    uint32_t last[kSets][kHeld], hoff[kHeld], hshift[kHeld];
    auto hold1 = [&](int set, int i, uint32_t k0) {
        if constexpr (!DIRECT) {
            const int8_t* p = (i < LM ? px : pw) + k0 + (int)hoff[i];
            __builtin_memcpy(&held[set][i], __builtin_assume_aligned(p, 4), 16);
            // the fifth word holds none of the bytes where the row starts on a word: the fourth again
            __builtin_memcpy(&last[set][i], __builtin_assume_aligned(p + (hshift[i] ? 16 : 12), 4), 4);
        }
    };
    auto put1 = [&](int set, int i, uint32_t buf) {
        if constexpr (!DIRECT) {
            const u32x4 h = held[set][i];
            const uint32_t t = hshift[i];
            *(u32x4*)(smem + buf * kStage + (i < LM ? 0 : BM * kI8BK) + (8 * NW * (i < LM ? i : i - LM) + wave * 8) * kI8BK +
                      16 * lane) =
                u32x4{__builtin_amdgcn_alignbyte(h.y, h.x, t), __builtin_amdgcn_alignbyte(h.z, h.y, t),
                      __builtin_amdgcn_alignbyte(h.w, h.z, t), __builtin_amdgcn_alignbyte(last[set][i], h.w, t)};
        }
    };
    if constexpr (!DIRECT) {
#pragma unroll
        for (int i = 0; i < LM + LN; ++i) {
            hshift[i] = (uint32_t)((uintptr_t)(i < LM ? px : pw) + off[i]) & 3u;
            hoff[i] = off[i] - hshift[i];                    // down to the word; -3 at the least
        }
    }

    const uint32_t frow = lane & 31u, fhalf = lane >> 5;
    const uint32_t fkey = i8_key(frow);                      // rows 32 apart have the same key
    const uint8_t* basex = smem + (wm * (BM / WM) + frow) * kI8BK;
    const uint8_t* basew = smem + (BM + wn * CW + frow) * kI8BK;
    i32x4 fr[2][TM + TN];                                    // fragments of w, then of x
    auto read1 = [&](int set, int f, uint32_t at) {
        fr[set][f] = f < TN ? *(const i32x4*)(basew + at + f * 32 * kI8BK)
                            : *(const i32x4*)(basex + at + (f - TN) * 32 * kI8BK);
    };
    auto place = [&](uint32_t buf, int kk) { return ((2u * kk + fhalf) ^ fkey) * 16u + buf * kStage; };
    i32x16 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = i32x16{};
    // One step of 32 bytes: the MFMAs of one fragment set with the other set's
    // reads and this step's share of moving a stage spread between them.  The
    // order is pinned: left to itself the compiler gathers the reads and waits.
    enum Move { kNone, kLoad, kPut };
    auto step = [&](int set, bool reads, uint32_t buf, int kk, Move move, uint32_t mbuf, uint32_t k0, int rset) {
        const uint32_t at = place(buf, kk);
        constexpr int kF = TM + TN, kM = TM * TN, kL = LM + LN;
#pragma unroll
        for (int m = 0; m < kM; ++m) {
            if (reads) {
#pragma unroll
                for (int f = (m * kF + kM - 1) / kM; f < ((m + 1) * kF + kM - 1) / kM; ++f)
                    if (f < kF) read1(set ^ 1, f, at);
            }
#pragma unroll
            for (int l = (m * kL) / kM; l < ((m + 1) * kL) / kM; ++l) {
                if (move == kPut) put1(rset, l, mbuf);
                if (move == kLoad) {
                    if constexpr (DIRECT) issue1(l, mbuf, k0);
                    else hold1(rset, l, k0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            acc[m / TN][m % TN] =
                __builtin_amdgcn_mfma_i32_32x32x32_i8(fr[set][m % TN], fr[set][TN + m / TN], acc[m / TN][m % TN], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    const int n = a.K / kI8BK;
    if (n > 0) {
        uint32_t buf = 0;
        int kt = 0;
        auto read_first = [&] {
#pragma unroll
            for (int f = 0; f < TM + TN; ++f) read1(0, f, place(0, 0));
        };
        if constexpr (DIRECT) {
            for (int i = 0; i < NS && i < n; ++i) issue(i, (uint32_t)i * kI8BK);
            // the first stage has landed when only the later ones' loads are out
            if (n >= NS) stage_barrier<(NS - 1) * (LM + LN)>();
            else stage_barrier<0>();
            read_first();
            // `left`: stages whose loads may be out when the next one has
            // landed; k0: the stage to load once this one is in registers
            auto stage = [&](auto left, bool more, bool loads, uint32_t k0) {
                const uint32_t next = buf + 1 == NS ? 0 : buf + 1;
                step(0, true, buf, 1, kNone, 0, 0, 0);
                step(1, true, buf, 2, kNone, 0, 0, 0);
                step(0, true, buf, 3, kNone, 0, 0, 0);
                // this stage's fragments are in registers, the next stage has landed
                stage_barrier<decltype(left)::value * (LM + LN)>();
                step(1, more, next, 0, loads ? kLoad : kNone, buf, k0, 0);
                buf = next;
            };
            for (; kt + NS < n; ++kt) stage(std::integral_constant<int, NS - 2>{}, true, true, (uint32_t)(kt + NS) * kI8BK);
            for (; kt + 1 < n; ++kt) stage(std::integral_constant<int, 0>{}, true, false, 0);
            stage(std::integral_constant<int, 0>{}, false, false, 0);
        } else {
            // stage s waits in set s % NR; the next stage moves from its set
            // to LDS, the set takes the stage NR further on
            auto hold = [&](int s) {
#pragma unroll
                for (int i = 0; i < LM + LN; ++i) hold1(s % NR, i, (uint32_t)s * kI8BK);
                __builtin_amdgcn_sched_barrier(0);           // set by set: they are waited for in this order
            };
            hold(0);
#pragma unroll
            for (int i = 0; i < LM + LN; ++i) put1(0, i, 0);
            auto stage = [&](int rset, bool more, bool loads, int at) {
                step(0, true, buf, 1, more ? kPut : kNone, buf ^ 1u, 0, rset);
                step(1, true, buf, 2, loads ? kLoad : kNone, 0, (uint32_t)(at + 1 + NR) * kI8BK, rset);
                step(0, true, buf, 3, kNone, 0, 0, 0);
                stage_barrier<63>();
                step(1, more, buf ^ 1u, 0, kNone, 0, 0, 0);
                buf ^= 1u;
            };
            // the long run starts from loads without a condition: with one, the
            // compiler cannot count what is on its way and waits for all of it
            if (2 * NR < n) {
#pragma unroll
                for (int s = 1; s <= NR; ++s) hold(s);
                stage_barrier<63>();
                read_first();
                for (; kt + 2 * NR < n; kt += NR) {
#pragma unroll
                    for (int r = 0; r < NR; ++r) stage((r + 1) % NR, true, true, kt + r);
                }
            } else {
#pragma unroll
                for (int s = 1; s <= NR; ++s)
                    if (s < n) hold(s);
                stage_barrier<63>();
                read_first();
            }
            for (; kt < n; kt += NR) {
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    if (kt + r < n) stage((r + 1) % NR, kt + r + 1 < n, kt + r + 1 + NR < n, kt + r);
            }
        }
    }
    // what is left of K, through registers: bytes past K are zeros
    if (n * kI8BK < a.K) {
        __syncthreads();
        for (uint32_t i = tid; i < (BM + BN) * 8; i += NT) {
            const uint32_t r = i >> 3, c = i & 7u;
            const bool isx = r < BM;
            const uint32_t q = isx ? r : r - BM;
            i32x4 v = {0, 0, 0, 0};
            if ((int)q < (isx ? rows_m : rows_n))
                v = ld_codes16((isx ? px + (size_t)q * ldx : pw + (size_t)q * ldw), n * kI8BK + 16 * (int)c, a.K);
            *(i32x4*)(smem + r * kI8BK + ((c ^ i8_key(q)) * 16u)) = v;
        }
        __syncthreads();
#pragma unroll
        for (int f = 0; f < TM + TN; ++f) read1(0, f, place(0, 0));
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) step(kk & 1, kk < 3, 0, kk + 1, kNone, 0, 0, 0);
    }
    __syncthreads();

    // Epilogue, wave by wave: 32 rows of sums through the wave's own slice of
    // LDS, read back with a lane on fixed columns (its scales stay in
    // registers) and stored as runs of CW columns.
    int* slice = (int*)smem + wave * 32 * kPitch;
    const bool vec = (((uintptr_t)a.y | (uint64_t)(a.ldy * (a.bf16 ? 2 : 4))) & 15u) == 0;
    auto store = [&](auto width) {
        constexpr int W = decltype(width)::value;            // columns of a lane: 16 bytes of y
        constexpr int kLanes = CW / W, kStep = 64 / kLanes;  // lanes of a row, rows of a pass
        const uint32_t col = (lane % kLanes) * W;
        const int64_t n = n0 + wn * CW + col;
        float sw[W], bias[W];
#pragma unroll
        for (int e = 0; e < W; ++e) {
            sw[e] = n + e < a.N ? a.sw[n + e] : 0.0f;
            bias[e] = a.bias && n + e < a.N ? a.bias[n + e] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            wave_lds_fence();
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *(i32x4*)(slice + frow * kPitch + 32 * j + 8 * q + 4 * fhalf) =
                        i32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
            wave_lds_fence();
#pragma unroll
            for (int p = 0; p < 32 / kStep; ++p) {
                const uint32_t r = p * kStep + lane / kLanes;
                const int64_t m = m0 + wm * (BM / WM) + 32 * i + r;
                if (m >= a.M || n >= a.N) continue;
                const float sx = a.sx[m];
                float v[W];
#pragma unroll
                for (int e = 0; e < W; ++e) v[e] = gemm_i8_value(slice[r * kPitch + col + e], sx, sw[e], a.bias, bias[e]);
                u32x4 u;                                     // 16 bytes of y
                if constexpr (W == 8) {
                    bf16x2 o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[e] = bf16x2{(__bf16)v[2 * e], (__bf16)v[2 * e + 1]};
                    __builtin_memcpy(&u, o, 16);
                } else {
                    __builtin_memcpy(&u, v, 16);
                }
                char* to = (char*)a.y + (m * a.ldy + n) * (16 / W);
                if (vec && n + W <= a.N) {
                    *(u32x4*)to = u;
                } else if (n + W <= a.N) {                   // rows at any place (4096 x 4095 x 1024: 27 us, 47 by elements)
                    __builtin_memcpy(to, &u, 16);
                } else {
#pragma unroll
                    for (int e = 0; e < W; ++e)
                        if (n + e < a.N) st_elem(a.y, a.bf16, m * a.ldy + n + e, v[e]);
                }
            }
        }
    };
    if (a.bf16) store(std::integral_constant<int, 8>{});
    else store(std::integral_constant<int, 4>{});
}

// ------------------------------------------------------------- few tokens --
//
// With few tokens the product is one pass over the weight, so nothing goes
// through LDS on the way in: a block of 8 waves takes 16 channels, each wave
// an eighth of K, and a lane's 16-byte load is its MFMA operand (16 rows x 64
// bytes per instruction).  The eight partial sums meet in LDS; integer sums
// are exact, so the split changes nothing.  Up to 16 MT tokens.
//
// Bound by the weight's way in: with eight weights in turn 1 x 4096 x 4096 takes
// 6.5 us, 2.6 TB/s over a call with its launch, and 8 x 8192 x 8192 17.3 us,
// 3.9 TB/s; with one that stays in cache 5.1 and 15.3.  All 64 KB that a CU
// has to read are asked for at once.
//
// XKIND 0 takes codes; 1 (bf16) and 2 (fp32) take up to FM tokens of
// activations, held in registers in C chunks of 8 a thread, and every block
// quantizes them into LDS while its first weight loads are on their way: one
// launch for the whole layer, the tokens coming from L2.

constexpr int kFewWaves = 8;
constexpr int kFewThreads = 64 * kFewWaves;
constexpr int kFewDepth = 8;                                 // weight loads of a wave in flight

struct FewArgs {
    GemmI8Args g;
    const void* xf;          // XKIND > 0: activations, rows of g.ldx
    int pitch;               // bytes of a token's codes in LDS
};

// whole steps of 64 codes, and 16 bytes that shift the tokens' banks
constexpr int few_pitch(int K) { return (K + 63) / 64 * 64 + 16; }

// 16 codes on their way to registers.  SHIFT: the row may start between two
// words; the words that hold the codes are loaded and shifted together (8 x
// 4096 x 4096: 7.7 us, as 16-byte loads at odd addresses 14.4, aligned 5.7).
template <bool SHIFT>
struct Codes16 {
    u32x4 v;
    uint32_t last[1];
    __device__ __forceinline__ void load(const int8_t* p)
    {
        if constexpr (SHIFT) {
            const uint32_t t = (uint32_t)(uintptr_t)p & 3u;
            __builtin_memcpy(&v, __builtin_assume_aligned(p - t, 4), 16);
            // the fifth word holds none of the codes where they start on a word: the fourth again
            __builtin_memcpy(last, __builtin_assume_aligned(p - t + (t ? 16 : 12), 4), 4);
        } else {
            __builtin_memcpy(&v, __builtin_assume_aligned(p, 4), 16);
        }
    }
    __device__ __forceinline__ i32x4 get(uint32_t t) const   // t: the address, or its two low bits
    {
        if constexpr (SHIFT)
            return i32x4{(int)__builtin_amdgcn_alignbyte(v.y, v.x, t), (int)__builtin_amdgcn_alignbyte(v.z, v.y, t),
                         (int)__builtin_amdgcn_alignbyte(v.w, v.z, t), (int)__builtin_amdgcn_alignbyte(last[0], v.w, t)};
        else
            return i32x4{(int)v.x, (int)v.y, (int)v.z, (int)v.w};
    }
};

template <int MT, int XKIND, int FM, int C, bool SHIFT>
__global__ __launch_bounds__(kFewThreads) void gemm_i8_few_kernel(const FewArgs a)
{
    extern __shared__ __align__(16) uint8_t few_lds[];
    __shared__ float few_scale[FM];
    __shared__ uint32_t few_max[kFewWaves][FM];
    const GemmI8Args& g = a.g;
    const uint32_t tid = threadIdx.x, lane = tid & 63u, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t row = lane & 15u, chunk = (lane >> 4) * 16u;
    const int M = (int)g.M;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int8_t* wr = g.w + min(n0 + row, g.N - 1) * g.ldw + chunk;

    // this wave's steps of 64 bytes
    const int steps = (g.K + 63) / 64;
    const int each = (steps + kFewWaves - 1) / kFewWaves;
    const int s0 = min(steps, (int)wave * each), s1 = min(steps, s0 + each);
    const int full = max(s0, min(s1, g.K / 64));             // up to here the steps lie inside K
    Raw8<XKIND != 2> raw[FM][C];
    if constexpr (XKIND > 0) {
#pragma unroll
        for (int m = 0; m < FM; ++m)
#pragma unroll
            for (int j = 0; j < C; ++j)
                raw[m][j] = ld_raw8<XKIND == 1, true>(a.xf, m * g.ldx, 8 * ((int)tid + kFewThreads * j), m < M ? g.K : 0);
    }
    Codes16<SHIFT> fw[kFewDepth];
    const uint32_t tw = (uint32_t)(uintptr_t)wr;             // steps of 64 keep a row's place in its words
    auto load_w = [&](int s) {
#pragma unroll
        for (int i = 0; i < kFewDepth; ++i)
            if (s + i < full) fw[i].load(wr + (int64_t)(s + i) * 64);
    };
    load_w(s0);

    if constexpr (XKIND > 0) {
#pragma unroll
        for (int m = 0; m < FM; ++m) {
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) top = max(top, abs_bits(raw_get(raw[m][j], e)));
            top = wave_max_u32(top);
            if (lane == 0) few_max[wave][m] = top;
        }
        __syncthreads();
#pragma unroll
        for (int m = 0; m < FM; ++m) {
            if (m >= M) continue;
            uint32_t top = 0;
#pragma unroll
            for (int w = 0; w < kFewWaves; ++w) top = max(top, few_max[w][m]);
            const TokenScale sc = token_scale(top);
            if (tid == 0) few_scale[m] = sc.scale;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const int k = 8 * ((int)tid + kFewThreads * j);
                if (k >= a.pitch - 16) continue;             // codes past K up to the last step are zeros
                uint32_t c[2] = {0, 0};
#pragma unroll
                for (int e = 0; e < 8; ++e) c[e / 4] |= (uint32_t)(token_code(raw_get(raw[m][j], e), sc.inv) & 255) << (8 * (e & 3));
                *(u32x2*)(few_lds + m * a.pitch + k) = u32x2{c[0], c[1]};
            }
        }
        __syncthreads();
    }

    i32x4 acc[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = i32x4{0, 0, 0, 0};
    // A lane past the last token repeats it: its sums are not stored, and a
    // load without a condition can be on its way with all the others.
    const int8_t* xr[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int m = min(16 * t + (int)row, M - 1);
        xr[t] = XKIND > 0 ? (const int8_t*)few_lds + m * a.pitch : g.x + m * g.ldx;
    }
    constexpr bool XSHIFT = SHIFT && XKIND == 0;
    auto x_load = [&](Codes16<XSHIFT>& f, int t, int s) {
        if constexpr (XKIND > 0) f.v = *(const u32x4*)(xr[t] + s * 64 + chunk);
        else f.load(xr[t] + (int64_t)s * 64 + chunk);
    };
    auto x_place = [&](int t) { return (uint32_t)(uintptr_t)xr[t]; };
    int s = s0;
    for (; s + kFewDepth <= full; s += kFewDepth) {
        Codes16<XSHIFT> fx[MT][kFewDepth];
#pragma unroll
        for (int i = 0; i < kFewDepth; ++i)
#pragma unroll
            for (int t = 0; t < MT; ++t) x_load(fx[t][i], t, s + i);
#pragma unroll
        for (int i = 0; i < kFewDepth; ++i) {
            const i32x4 w = fw[i].get(tw);
#pragma unroll
            for (int t = 0; t < MT; ++t)
                acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, fx[t][i].get(x_place(t)), acc[t], 0, 0, 0);
        }
        load_w(s + kFewDepth);
    }
#pragma unroll
    for (int i = 0; i < kFewDepth; ++i) {
        if (s + i < full) {
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                Codes16<XSHIFT> f;
                x_load(f, t, s + i);
                acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[i].get(tw), f.get(x_place(t)), acc[t], 0, 0, 0);
            }
        }
    }
    if (full < s1) {                                         // the step that K ends in
        const i32x4 w = ld_codes16(wr - chunk, full * 64 + (int)chunk, g.K);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const i32x4 v = XKIND > 0 ? *(const i32x4*)(xr[t] + full * 64 + chunk)
                                      : ld_codes16(xr[t], full * 64 + (int)chunk, g.K);
            acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w, v, acc[t], 0, 0, 0);
        }
    }

    // sum over the waves: lane l of tile t holds channels 4 (l / 16) .. + 3 of token 16 t + l % 16
    __syncthreads();
    i32x4* part = (i32x4*)few_lds;
#pragma unroll
    for (int t = 0; t < MT; ++t) part[(wave * MT + t) * 64 + lane] = acc[t];
    __syncthreads();
    for (uint32_t i = tid; i < 64 * MT; i += kFewThreads) {
        i32x4 v = part[i];
#pragma unroll
        for (int w = 1; w < kFewWaves; ++w) {
            const i32x4 o = part[w * MT * 64 + i];
            v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
        }
        const int m = 16 * (int)(i >> 6) + (int)(i & 15u);
        if (m >= M) continue;
        const int64_t n = n0 + 4 * ((i & 63u) >> 4);
        const float sx = XKIND > 0 ? few_scale[m] : g.sx[m];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < g.N)
                st_elem(g.y, g.bf16, m * g.ldy + n + e,
                        gemm_i8_value(v[e], sx, g.sw[n + e], g.bias, g.bias ? g.bias[n + e] : 0.0f));
    }
}

}  // namespace echo
