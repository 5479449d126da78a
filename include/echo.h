/*
 * echo.h — C ABI of libecho: the per-call hot path of Echo's
 * error-compensated low-bit all-reduce, on one MI355X (gfx950).
 *
 * Sources: "Echo: Error-Compensated 4-Bit Tensor-Parallel Communication for
 * LLM Training and Inference" (arXiv 2610.14277), paper card: abstract,
 * Fig. 1, Fig. 2(a)/(b), Table 8, appendix Fig. 4; and the PhantomByte article
 * "Your All-Reduce Is 4x Overpriced: Echo's 4-Bit Error-Feedback Trick for
 * Tensor-Parallel Training", section "The cancellation rule".
 *
 * The problem: P tensor-parallel ranks each hold a partial sum x_r of n
 * bfloat16 values; the all-reduce returns sum_r x_r to every rank.  Echo
 * splits the message into P equal contiguous segments, segment s owned by
 * rank s.  Each rank adds its compensation, quantizes the P-1 segments that
 * belong to other ranks and sends those codes to the segments' owners; an
 * owner decodes the P-1 copies it received, adds its own copy (never
 * quantized) in fp32 and quantizes the total a single time; every rank
 * decodes that same code.  The errors the sum reveals feed a
 * compensator whose output is added at the next call.
 *
 * Here the P ranks are P sets of buffers on one GPU: "push" and "gather"
 * move no bytes between devices; each simulated rank still performs its own
 * reads and writes.
 *
 * Conventions for every call:
 *  - Pointers marked (device) are device memory, (host) are host memory.  The
 *    caller owns every buffer and keeps it alive until the enqueued work is
 *    done.  The library never allocates or frees device memory.
 *  - `stream` is a hipStream_t (NULL = the null stream).  Calls only enqueue;
 *    they do not synchronize.
 *  - Arguments are checked on the host before anything is enqueued; a call
 *    that returns an error other than ECHO_EHIP has enqueued nothing.
 *  - Data pointers must be 16-byte aligned (ECHO_EALIGN otherwise); the block
 *    operators at the end have conventions of their own for this and for
 *    non-finite inputs.
 *  - Messages: n elements per rank, 0 <= n <= 2^34, n a multiple of P*group.
 *    S = n / P is the segment length.  Tiles are element ranges *inside each
 *    segment*: [tile_begin, tile_begin + tile_len), both multiples of group,
 *    tile_begin + tile_len <= S.  (0, S) means whole segments.
 *  - bits is 4 or 8; group is 128 or 256 (ECHO_EUNSUP otherwise).  P is 1..8.
 *  - Codes: unsigned, 0 .. 2^bits - 1.  bits = 4: element i's code is in byte
 *    i/2, the low nibble when i is even; bits = 8: byte i.  Code arrays are
 *    message-shaped: n*bits/8 bytes, segment s at byte offset s*S*bits/8.
 *  - Per-group parameters: one echo_qparam per group of `group` consecutive
 *    message elements (n/group entries, message-shaped): IEEE binary16 scale s
 *    and binary16 zero point z.  Decoding is v = (q - z) * s in fp32: exact
 *    when z is an integer (the zero-aware quantizer and the symmetric-grid
 *    ablation); the naive-zero-point ablation's z carries a fraction, so
 *    there q - z may round.
 *  - Non-finite inputs give unspecified (but memory-safe) results.
 *  - Thread safety: calls are reentrant.  Calls that write the same buffers
 *    must be ordered by the caller.
 */
#ifndef ECHO_H
#define ECHO_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum echo_status {
    ECHO_OK = 0,
    ECHO_EINVAL = -1, /* null required pointer, bad P/rank/owner/constants */
    ECHO_EALIGN = -2, /* a data pointer is not 16-byte aligned (block operators: not aligned to its element) */
    ECHO_EUNSUP = -3, /* bits not 4/8, group not 128/256, unknown dtype */
    ECHO_ESHAPE = -4, /* n or tile not a valid multiple / out of range */
    ECHO_EHIP = -5,   /* a HIP launch or runtime call failed; see echo_last_hip_error */
    ECHO_ETOOBIG = -6 /* echo_allreduce_sim_noalloc: the message needs more workspace than
                         echo_noalloc_scratch_bytes() */
};

enum echo_out_dtype { ECHO_OUT_F32 = 0, ECHO_OUT_BF16 = 1 };

/* element types of the block operators (same values as echo_out_dtype) */
enum echo_dtype { ECHO_F32 = 0, ECHO_BF16 = 1, ECHO_I8 = 2, ECHO_I4 = 3 };

/* flags for echo_quantize_ef / echo_reduce_segment / echo_gemm_quantize_ef
 * (and echo_sim_args.quant for the two quantizer bits) */
enum {
    ECHO_ERR_NEGATED = 1,      /* write -e (the next call's compensation) instead of e */
    ECHO_QUANT_NAIVE = 2,      /* Table 8 ablation: naive zero point */
    ECHO_QUANT_SYMMETRIC = 4,  /* Table 8 ablation: symmetric grid */
    ECHO_X_ALL = 8,            /* echo_gemm_quantize_ef only: write x for every segment */
    ECHO_QUANT_MSE = 16        /* full method with its zero point searched for the least squared error */
};

#define ECHO_MAX_P 8

typedef struct echo_qparam {
    uint16_t scale_f16; /* binary16 bits of s */
    uint16_t zero_f16;  /* binary16 bits of the zero point z (an integer except
                           for the naive-zero-point ablation) */
} echo_qparam;

/*
 * echo_quantize_ef — entry pass and push quantization for one rank.
 * Paper card Fig. 2(a) and Fig. 4 (each rank quantizes the segments it does
 * not own, keeps its own); article "The cancellation rule" (the compensation
 * is added in the entry pass; parameters are half precision per group);
 * Table 8 (zero-aware asymmetric quantizer, g = 128).
 *
 * For every segment s != rank and every group of the tile inside it:
 *   u = float(x) + comp            (u = float(x) when comp is NULL)
 *   lo = min(0, min u), hi = max(0, max u)
 *   s = binary16((hi - lo) / (2^bits - 1)), round to nearest even; a zero
 *       result becomes 2^-24 and an infinite one 65504; hi == lo (an all-zero
 *       group) gives s = +0, z = 0 and all codes 0
 *   z = clamp(rint(-lo * (1/s)), 0, 2^bits - 1)
 *   q = clamp(rint(u * (1/s)) + z, 0, 2^bits - 1)
 *   err = (q - z) * s - u          (or its negation with ECHO_ERR_NEGATED)
 * All float operations are single IEEE fp32 operations (no contraction);
 * 1/s and the scale division are correctly rounded; rint rounds half to even.
 *
 * The quantizer above is the full method's (zero-aware asymmetric, Table 8).
 * The flag bits select one of Table 8's ablations instead (same parameter
 * word, same decode v = (q - z) * s):
 *   ECHO_QUANT_NAIVE      lo = min u, hi = max u (no widening to 0);
 *                         s as above; z = binary16((0 - lo) * (1/s)), a real
 *                         value (+0 when the minimum is a zero of either sign;
 *                         an overflow becomes +-65504); q = clamp(rint(u *
 *                         (1/s) + z), 0, Qm); hi == lo gives s = +0, z = 0,
 *                         codes 0.
 *   ECHO_QUANT_SYMMETRIC  a = max |u|; s = binary16(a / (2^(bits-1) - 1))
 *                         with the clamps above; z = 2^(bits-1);
 *                         q = clamp(rint(u * (1/s)) + z, 0, Qm); a == 0 gives
 *                         s = +0 and all codes z.
 * ECHO_QUANT_MSE keeps the full method's s and codes rule and searches the
 * integer zero point instead of taking the closed form: the z in [0, Qm]
 * minimizing sum_i (clamp(rint(t_i) + z, 0, Qm) - z - t_i)^2 with
 * t_i = u_i * (1/s), the smallest z on ties (it differs from the closed form
 * only where the rounded codes span more than 2^bits levels).
 * Setting more than one quantizer bit is ECHO_EINVAL.
 *
 *   x_bf16 (device, in)   bfloat16 bits [n] of this rank's partial sums
 *   comp   (device, in)   fp32 [n] compensation, or NULL (no feedback)
 *   codes  (device, out)  this rank's push codes (message-shaped)
 *   params (device, out)  this rank's push parameters (message-shaped)
 *   err    (device, out)  fp32 [n] revealed error, or NULL.  May alias comp:
 *                         each element is read before it is overwritten.
 * Elements of segment `rank` and outside the tile are not touched.
 */
int echo_quantize_ef(const uint16_t* x_bf16, const float* comp, int64_t n, int P, int rank,
                     int64_t tile_begin, int64_t tile_len, int bits, int group,
                     uint8_t* codes, echo_qparam* params, float* err, int flags, void* stream);

/*
 * echo_reduce_segment — the owner's high-precision sum and single
 * requantization.  Paper card Fig. 2(a) (decode of the peers' codes, the
 * owner's own copy added without quantization, one quantization of the total
 * before the all-gather), Fig. 4, abstract (the sum reveals each injected
 * error).
 *
 * For every group of segment `owner` inside the tile:
 *   t_j = float(own_x) + own_comp       when j == owner (no quantization)
 *   t_j = (q_j - z_j) * s_j              from peer j's push codes otherwise
 *   acc = t_0 + t_1 + ... + t_{P-1}      in fp32, left to right in rank order
 *   sum codes / params = Q(acc)          (the quantizer of echo_quantize_ef)
 *   own_err = (q - z) * s - acc          (or its negation with ECHO_ERR_NEGATED)
 *
 *   own_x_bf16, own_comp (device, in)  the owner's x and comp (comp nullable)
 *   peer_codes, peer_params (host arrays of P device pointers, in)
 *                                      each rank's push codes/params, made by
 *                                      echo_quantize_ef with the same
 *                                      quantizer flag; entry [owner] is not
 *                                      read and may be NULL
 *   sum_codes, sum_params (device, out) message-shaped; only segment `owner`
 *                                      inside the tile is written
 *   own_err (device, out, nullable)    fp32 [n]; may alias own_comp
 */
int echo_reduce_segment(const uint16_t* own_x_bf16, const float* own_comp,
                        const uint8_t* const* peer_codes, const echo_qparam* const* peer_params,
                        int P, int owner, int64_t n, int64_t tile_begin, int64_t tile_len,
                        int bits, int group, uint8_t* sum_codes, echo_qparam* sum_params,
                        float* own_err, int flags, void* stream);

/*
 * echo_gather_dequant — quantized all-gather and tail decode for one rank.
 * Paper card Fig. 2(a) (every rank, the owner included, decodes the same
 * code, so all outputs are identical), Fig. 4.
 *
 * For every segment and every element of the tile inside it:
 *   out[i] = (q_i - z) * s   as fp32, or rounded to bfloat16 (nearest even)
 *
 *   sum_codes, sum_params (device, in)  the owners' sum codes (message-shaped)
 *   out (device, out)  fp32 [n] (ECHO_OUT_F32) or bfloat16 bits [n] (ECHO_OUT_BF16)
 */
int echo_gather_dequant(const uint8_t* sum_codes, const echo_qparam* sum_params, int64_t n,
                        int64_t tile_begin, int64_t tile_len, int P, int bits, int group,
                        void* out, int out_dtype, void* stream);

/*
 * echo_compensate — the two-timescale compensator update, elementwise.
 * Paper card abstract (a revealed error is returned in a later call, which
 * cancels it); article "The cancellation rule" (a two-timescale compensator,
 * updated off the critical path while the next matmul runs).  The
 * pages give no equation; the reading is an error debt with a fast fraction
 * alpha returned at the next call and a slow memory M released at rate beta:
 *   comp_next = -(alpha*e + beta*M)
 *   M         = (1-beta)*M + (1-alpha)*e
 * (products rounded, then the sum, then the negation).  With slow == NULL
 * (beta must be 0): comp_next = -(alpha*e); alpha = 1 is classic error feedback.
 *
 *   err (device, in)        fp32 [n] revealed errors of the last call
 *   comp_next (device, out) fp32 [n]; may alias err
 *   slow (device, in/out)   fp32 [n] slow memory M, or NULL
 * Constraints: 0 < alpha <= 1, 0 <= beta <= 1, beta > 0 iff slow != NULL,
 * alpha < 1 requires beta > 0 (ECHO_EINVAL otherwise).
 */
int echo_compensate(const float* err, float* comp_next, float* slow, int64_t n,
                    float alpha, float beta, void* stream);

/*
 * echo_gemm_quantize_ef — one rank's row-parallel matmul with the entry pass
 * and push quantization fused into its epilogue.  Paper card Fig. 2(a) (each
 * rank quantizes its partial sums for the segments owned by other ranks);
 * article "The cancellation rule" (the compensator is folded into the entry
 * pass, beside the matmul, and the results stay as they were).
 *
 * Computes this rank's partial sums x = bf16(A W^T), i.e.
 *   x[m*N + j] = bfloat16(sum_k A[m][k] * W[j][k])   (fp32 accumulation,
 *                                                     round to nearest even)
 * and then does exactly what echo_quantize_ef(x, comp, M*N, P, rank, 0,
 * M*N/P, bits, group, codes, params, err, flags) does, without writing x for
 * the pushed segments: the message is x in row-major order, segment s is
 * rows [s*M/P, (s+1)*M/P), one group is `group` consecutive columns of a row.
 * The rank's own segment of x is written to x_out (bf16), for the owner
 * reduce; with ECHO_X_ALL, x_out receives every segment.  The fp32 sum order
 * is the kernel's own (K in steps of 16, MFMA accumulation), so x matches a
 * separate GEMM only up to fp32 rounding of the sum; everything after x is
 * bit-exact.
 * Performance: measured at a Llama-3-8B MLP down projection at TP = 4
 * (M = N = 4096, K = 3584), this call is usually slower than a library
 * matmul (hipBLASLt) followed by echo_quantize_ef, by about 3 to 10 %
 * depending on the GPU (on one it was 3 % faster): its matmul core is
 * slower than the library's, and its epilogue (the push) cannot overlap the
 * matrix cores when every CU holds one output tile.  Prefer the separate
 * pair where speed matters.
 *
 *   a_bf16 (device, in)   bfloat16 bits [M][K], row-major (K contiguous)
 *   w_bf16 (device, in)   bfloat16 bits [N][K], row-major (K contiguous): the
 *                         weight of y = a w^T
 *   comp   (device, in)   fp32 [M*N] compensation, or NULL (no feedback)
 *   codes, params, err    as for echo_quantize_ef (message-shaped; err may
 *                         alias comp or be NULL)
 *   x_out  (device, out)  bfloat16 bits [M*N]; rows of segment `rank` (all
 *                         rows with ECHO_X_ALL) are written, others untouched
 * Constraints: group 128 or 256 (ECHO_EUNSUP otherwise); M and N multiples of
 * 256, K a positive multiple of 64 below 2^22, M a multiple of P with
 * M/P a multiple of 16, M*N <= 2^34 (ECHO_ESHAPE); M or N of 0 enqueues nothing.  Flags: those
 * of echo_quantize_ef and ECHO_X_ALL.
 * Pointers as for echo_quantize_ef (codes and params may be NULL when P == 1,
 * as nothing is pushed), plus a_bf16, w_bf16 and x_out required.
 */
int echo_gemm_quantize_ef(const uint16_t* a_bf16, const uint16_t* w_bf16, int64_t M, int64_t N,
                          int64_t K, const float* comp, int P, int rank, int bits, int group,
                          uint8_t* codes, echo_qparam* params, float* err, uint16_t* x_out,
                          int flags, void* stream);

/*
 * echo_allreduce_sim — one whole call for P simulated ranks: push, owner
 * reduce, gather, tail decode and (if on) the compensator update, with each
 * segment split into `tiles` tiles whose stages overlap on several streams.
 * Paper card Fig. 2(b) (the stages of successive tiles overlap in time;
 * events order the work inside a GPU).
 *
 * Stage k of every tile runs on streams[k % nstreams] (push 0, reduce 1,
 * tail 2, compensator 3); events order tile t's reduce after its pushes and
 * its tail after its reduce.  Tile t's tail is enqueued after tile t+1's
 * push, so with two streams (the tail sharing the push's stream) the reduce
 * of a tile still runs beside the push of the next.  The gather moves no bytes here: the tail reads
 * the owners' sum codes directly.  All streams start after the work already
 * enqueued on streams[0], and streams[0] waits for all of them before the
 * call returns, so the caller may treat the call as enqueued on streams[0].
 * streams may be NULL (null stream only).  Results do not depend on tiles or
 * streams (bit for bit).
 *
 * One tile and at most 2^20 elements per rank: the whole call is one launch
 * on streams[0] (each block takes one 512-element chunk of one segment, and
 * its four wavefronts split the ranks: they push their ranks' copies, the
 * owner's wavefront reduces, and each decodes the sum into its ranks'
 * outputs; every stage still writes and reads its own buffers), followed by
 * echo_compensate when err[r] are given.
 * Such a call is bound by launch latency, and one launch instead of one per
 * stage cuts it; the results are the same bit for bit.
 *
 * Feedback (ef = 1): every rank's comp is added at the entry pass.  With
 * err[r] == NULL for every rank the update is fused into the push and reduce
 * kernels: they write -e straight into comp (alpha = 1, beta = 0, classic
 * error feedback) or apply the two-timescale update to comp and slow in place
 * (beta > 0).  Both are bit-identical to writing e and running
 * echo_compensate, which is what happens when err[r] are given: err[r]
 * receives e, and echo_compensate turns it into comp[r] (and slow[r]) after
 * the call's last reduce.
 *
 * The workspace (device, caller-allocated, >= echo_allreduce_sim_workspace_bytes)
 * holds every rank's push codes/params and the sum codes/params.
 */
typedef struct echo_sim_args {
    int P;          /* ranks, 1..8 */
    int bits;       /* 4 or 8 */
    int group;      /* 128 or 256 */
    int tiles;      /* tiles per segment, >= 1 (capped at S/group and at 4096) */
    int out_dtype;  /* ECHO_OUT_F32 or ECHO_OUT_BF16 */
    int ef;         /* 0: no compensation; 1: compensation on */
    int quant;      /* 0 (zero-aware), ECHO_QUANT_NAIVE, ECHO_QUANT_SYMMETRIC or ECHO_QUANT_MSE */
    float alpha;    /* fast fraction, 0 < alpha <= 1 */
    float beta;     /* slow release rate, 0 <= beta <= 1 */
    int64_t n;      /* elements per rank */
    const uint16_t* x[ECHO_MAX_P]; /* (device) bf16 bits [n] per rank */
    float* comp[ECHO_MAX_P];       /* (device) fp32 [n] per rank (ef = 1) */
    float* slow[ECHO_MAX_P];       /* (device) fp32 [n] per rank (beta > 0) */
    float* err[ECHO_MAX_P];        /* (device) fp32 [n] per rank, or NULL (update fused) */
    void* out[ECHO_MAX_P];         /* (device) [n] fp32 or bf16 bits per rank */
    void* workspace;               /* (device) */
    size_t workspace_bytes;
} echo_sim_args;

/* Bytes of workspace echo_allreduce_sim needs; 0 for invalid arguments. */
size_t echo_allreduce_sim_workspace_bytes(int P, int64_t n, int bits, int group);

/* streams: host array of nstreams hipStream_t handles, or NULL. */
int echo_allreduce_sim(const echo_sim_args* args, void* const* streams, int nstreams);

/*
 * echo_allreduce_sim_noalloc — echo_allreduce_sim for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation).  It allocates nothing: the push and sum
 * codes go to a static device array of echo_noalloc_scratch_bytes() bytes
 * (64 MiB) that the library holds on every device it runs on until the
 * process ends; args->workspace and args->workspace_bytes are ignored.  Every
 * stage runs on `stream` (hipStream_t, NULL = the null stream), tile after
 * tile, so no events are created either; results are those of
 * echo_allreduce_sim, bit for bit.  The first call on a device looks up the
 * array's device address (hipGetSymbolAddress) and keeps it.
 *
 * Errors: those of echo_allreduce_sim (except the workspace checks), and
 * ECHO_ETOOBIG, with nothing enqueued, when
 * echo_allreduce_sim_workspace_bytes(P, n, bits, group) exceeds the array:
 * at 4-bit codes and g = 128 that is n above about 25 million elements per
 * rank for P = 4.  Calls on one device share the array: calls that overlap
 * in time on one device race and must be ordered by the caller (for example
 * by issuing them on one stream).  Nothing in the array needs clearing
 * between calls: every byte a call reads was written earlier in that call.
 */
int echo_allreduce_sim_noalloc(const echo_sim_args* args, void* stream);

/* Size in bytes of the static scratch array of echo_allreduce_sim_noalloc. */
size_t echo_noalloc_scratch_bytes(void);

/*
 * The block operators: what stands on both sides of the all-reduce in a
 * tensor-parallel block.  A row-parallel layer in 8-bit integers makes the
 * partial sums; the norms that close the block and open the next one take
 * the summed output.
 *
 * Conventions, beside those above:
 *  - A matrix is rows of contiguous elements at a distance of ld elements
 *    (ld >= the row's length; a single row's ld is not used).  Nothing
 *    outside the rows is written, and no aligned 4-byte word that holds none
 *    of a row is read.
 *  - Pointers need the alignment of their element type only (workspaces 16
 *    bytes); where the base and ld of every matrix of a call are multiples of
 *    16 bytes the call is fastest.
 *  - Non-finite values: what is normed, quantized or multiplied from a token
 *    that holds an infinity or a NaN is NaN throughout (8-bit codes are 0 with
 *    a scale of NaN), and so are that token's gradients; a residual sum has it
 *    where it stands.  No other token is touched (the sums over tokens in a
 *    backward pass take it up).  Finite values are normed by the formulas
 *    whatever their size, also where their squares leave fp32.
 *  - Inputs and outputs do not overlap except where a call says so.
 */

/*
 * echo_quantize_tokens — 8-bit codes and one scale for each token.
 *   a = max(max_k |x[t][k]|, 2^-100),  scales[t] = a / 127,
 *   codes[t][k] = rint(x[t][k] * (127 / a)), in [-127, 127]
 * in single IEEE fp32 operations, rint half to even.  A token with an
 * infinity or a NaN gets the scale NaN and codes 0.
 *
 *   x (device, in)       [T][K], ECHO_F32 or ECHO_BF16, rows at ldx
 *   codes (device, out)  [T][K] rows at ldq
 *   scales (device, out) [T]
 * Constraints: 0 <= K <= 131071, 0 <= T < 2^31 (ECHO_ESHAPE).
 */
int echo_quantize_tokens(const void* x, int64_t ldx, int x_dtype, int64_t T, int64_t K,
                         int8_t* codes, int64_t ldq, float* scales, void* stream);

/*
 * echo_gemm_int8 — product of 8-bit integers with a scale for each token and
 * each channel:
 *   y[m][n] = float(sum_k x[m][k] * w[n][k]) * sx[m] * sw[n] (+ bias[n])
 * The sum is exact (32-bit integers), so results depend on no order; it is
 * rounded to fp32, multiplied by sx and then by sw, and the bias is added,
 * each a single fp32 operation; a bf16 y is rounded once more.
 * With the codes of echo_quantize_tokens and a weight quantized by rows of
 * its [N][K] form this is the linear layer y = x w^T + bias; its partial sums
 * (ECHO_BF16, ldy = N) are the message of echo_quantize_ef and
 * echo_allreduce_sim.
 *
 *   x (device, in)   [M][K] codes, rows at ldx; any value of int8
 *   w (device, in)   [N][K] codes, rows at ldw
 *   sx, sw (device, in) [M], [N];  bias (device, in) fp32 [N] or NULL
 *   y (device, out)  [M][N], ECHO_F32 or ECHO_BF16, rows at ldy
 * Constraints: 0 <= K <= 131071 (the sum stays in 32 bits), M, N < 2^31,
 * and at most 2^31 - 1 tiles of 64 x 64 (ECHO_ESHAPE).  M or N of 0 enqueues
 * nothing; K of 0 gives y = bias (or 0).
 */
int echo_gemm_int8(const int8_t* x, int64_t ldx, const float* sx, const int8_t* w, int64_t ldw,
                   const float* sw, const float* bias, int64_t M, int64_t N, int64_t K, void* y,
                   int64_t ldy, int y_dtype, void* stream);

/*
 * echo_linear_int8 — echo_quantize_tokens of x followed by echo_gemm_int8, bit
 * for bit.  The workspace (device, 16-byte aligned, at least
 * echo_linear_int8_workspace_bytes) holds the codes and scales between the
 * two; it may be NULL where that function returns 0.
 */
size_t echo_linear_int8_workspace_bytes(int64_t M, int64_t N, int64_t K);
int echo_linear_int8(const void* x, int64_t ldx, int x_dtype, const int8_t* w, int64_t ldw,
                     const float* sw, const float* bias, int64_t M, int64_t N, int64_t K, void* y,
                     int64_t ldy, int y_dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * echo_block_norm — the norms that close one block and open the next, around
 * the gated, scaled residual sum.  For every token:
 *   z  = x * rsqrt(mean(x^2) + eps) * w_post   (post = 1; z = x for post = 0)
 *   r' = res_scale * r + block_scale * gate * z
 *   h  = r' * rsqrt(mean(r'^2) + eps) * w_pre
 * in fp32; r_out receives r', h the normed stream (rounded once, from the
 * unrounded r'), as fp32, bf16 or 8-bit codes with a scale for each token
 * (those of echo_quantize_tokens applied to the unrounded h).
 *
 * x is the block's output (the all-reduced sum), r the residual stream.  One
 * row of the gate serves gate_tokens consecutive tokens: 1 is a gate for each
 * token, the sequence length one for each sequence, T or more one for all;
 * the last row may serve fewer.  r NULL is a stream of zeros (the first
 * norm of a model: post = 0, x the embeddings), w_post, w_pre and gate NULL
 * are ones, r_out or h may be NULL (not both).  r_out may be r.  H of 0 writes
 * the scales of an 8-bit h (where h_scale is not NULL) and nothing else.
 * Constraints: T < 2^31, H <= 2^30 (ECHO_ESHAPE); eps > 0 and the scales
 * finite, w_post NULL where post = 0 (ECHO_EINVAL).
 */
typedef struct echo_norm_args {
    int64_t T, H;                                  /* tokens, width */
    int64_t ld_x, ld_r, ld_r_out, ld_h, ld_gate;   /* row distances in elements */
    int64_t gate_tokens;                           /* tokens of one gate row, >= 1 with a gate */
    int x_dtype, r_dtype, w_dtype;                 /* ECHO_F32 or ECHO_BF16; r_dtype also of r_out, w_dtype
                                                      of w_post, w_pre and gate */
    int h_dtype;                                   /* ECHO_F32, ECHO_BF16 or ECHO_I8 */
    int post;                                      /* 1: post norm, 0: none */
    float eps, res_scale, block_scale;
    const void* x;                                 /* (device) [T][H] */
    const void* r;                                 /* (device) [T][H] or NULL */
    const void* w_post;                            /* (device) [H] or NULL */
    const void* w_pre;                             /* (device) [H] or NULL */
    const void* gate;                              /* (device) [ceil(T / gate_tokens)][H] or NULL */
    void* r_out;                                   /* (device) [T][H] or NULL */
    void* h;                                       /* (device) [T][H] or NULL */
    float* h_scale;                                /* (device) [T], required for an ECHO_I8 h */
} echo_norm_args;

int echo_block_norm(const echo_norm_args* args, void* stream);

/*
 * echo_block_norm_backward — gradients of echo_block_norm.  args are the
 * forward call's (its r_out, h and h_scale are not used; r and x have to hold
 * what they held then, so keep r where the forward call wrote r_out over it).
 * The gradient of an 8-bit h is taken as that of the unquantized h.
 *
 *   dh (device, in)      [T][H] gradient of h, ECHO_F32 or ECHO_BF16, or NULL (zero)
 *   dr_out (device, in)  [T][H] gradient of r_out in r's type, or NULL (zero)
 *   dx, dr (device, out) [T][H] in x's and r's type, or NULL; dr may be dr_out
 *   dw_post, dw_pre (device, out) fp32 [H] or NULL: sums over all tokens
 *   dgate (device, out)  fp32 [ceil(T / gate_tokens)][H] or NULL: sums over
 *                        each gate row's tokens
 * The sums run in fp32 in a fixed order (equal inputs give equal bits).
 * The workspace (device, 16-byte aligned) has at least
 * echo_block_norm_backward_workspace_bytes bytes.  T of 0 writes zeros to
 * dw_post and dw_pre.  ECHO_EINVAL: both dh and dr_out NULL (T > 0), dgate
 * without a gate, dw_post without the post norm, dr without r.
 */
typedef struct echo_norm_grads {
    int64_t ld_dh, ld_dr_out, ld_dx, ld_dr, ld_dgate;
    int dh_dtype;
    const void* dh;
    const void* dr_out;
    void* dx;
    void* dr;
    float* dw_post;
    float* dw_pre;
    float* dgate;
    void* workspace;
    size_t workspace_bytes;
} echo_norm_grads;

size_t echo_block_norm_backward_workspace_bytes(int64_t T, int64_t H);
int echo_block_norm_backward(const echo_norm_args* args, const echo_norm_grads* grads, void* stream);

/*
 * Serving operators: a rank's step between the norm's output and the message
 * of the all-reduce with low-bit weights and a low-bit cache.  Conventions of
 * the block operators, and:
 *  - 4-bit codes lie two to a byte, the even element in the low nibble; a
 *    value is (q - z) * s with its group's echo_qparam, as everywhere above.
 *  - 4-bit codes and parameters are made by the full method's quantizer
 *    (echo_quantize_ef), bit for bit.  A group that holds an infinity or a NaN
 *    gets the scale NaN, the zero point 0 and codes 0.
 */

/*
 * echo_quantize_groups — 4-bit codes and parameters of every `group`
 * consecutive elements of a row; the last group of a row may be shorter.
 *
 *   x (device, in)       [T][K], ECHO_F32 or ECHO_BF16, rows at ldx
 *   codes (device, out)  [T][(K + 1) / 2] bytes, rows at ldq bytes; the high
 *                        nibble behind an odd K is 0
 *   params (device, out) [T][ceil(K / group)], rows at ldp, 4-byte aligned
 * Constraints: group 32, 64, 128 or 256 (ECHO_EUNSUP); 0 <= K <= 2^30,
 * 0 <= T < 2^31 (ECHO_ESHAPE).
 */
int echo_quantize_groups(const void* x, int64_t ldx, int x_dtype, int64_t T, int64_t K, int group, uint8_t* codes,
                         int64_t ldq, echo_qparam* params, int64_t ldp, void* stream);

/*
 * echo_linear_int4 — a linear layer with 4-bit weights, for few tokens:
 *   y[m][n] = sum_g s[n][g] * sum_{k in g} x[m][k] * (q[n][k] - z[n][g])  (+ bias[n])
 * The products are exact and summed in fp32, group by group; a group's sum
 * takes its scale in fp32, and a bf16 y is rounded once.  The order of the
 * sums is fixed: equal calls give equal bits.  z is an integer from 0 to 15
 * (what the quantizer above makes); other zero points round once, beside 16.
 * A token that holds an infinity or a NaN is NaN throughout.  It is made for
 * few tokens: every 64 tokens (32 in fp32) read the weight again.
 *
 *   x (device, in)      [M][K], ECHO_F32 or ECHO_BF16, rows at ldx
 *   w (device, in)      [N][(K + 1) / 2] bytes of codes, rows at ldw bytes
 *   params (device, in) [N][ceil(K / group)], rows at ldp
 *   bias (device, in)   fp32 [N] or NULL
 *   y (device, out)     [M][N], ECHO_F32 or ECHO_BF16, rows at ldy
 * Constraints: group as above; 0 <= K <= 2^30, M <= 2^21 - 32, M * K <= 2^36,
 * N < 2^31 and fewer than 2^23 tiles of 16 channels by 32 tokens (ECHO_ESHAPE).  M or N of 0 enqueues
 * nothing; K of 0 gives y = bias (or 0).  The workspace (device, 16-byte
 * aligned, at least echo_linear_int4_workspace_bytes) holds the tokens laid
 * out for the product; it may be NULL where that function returns 0.  Calls
 * that may overlap in time need one each.
 */
size_t echo_linear_int4_workspace_bytes(int64_t M, int64_t N, int64_t K, int group);
int echo_linear_int4(const void* x, int64_t ldx, int x_dtype, const uint8_t* w, int64_t ldw, const echo_qparam* params,
                     int64_t ldp, int group, const float* bias, int64_t M, int64_t N, int64_t K, void* y, int64_t ldy,
                     int y_dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * echo_cache — a paged cache of keys and values: `pages` pages of
 * `page_tokens` tokens, each token a row of `width` elements for each of
 * `heads` heads.  Element d of head h of the token in slot i of page p lies at
 *   p * ld_page + h * ld_head + i * ld_token + d
 * in k and in v (in elements; rows do not overlap).  Rows are
 *   ECHO_BF16  the values
 *   ECHO_I8    codes with an fp32 scale a row: those of echo_quantize_tokens
 *   ECHO_I4    codes with an echo_qparam a row: those of echo_quantize_groups
 *              with the row as its group
 * and a row's scale or parameter lies at p * ld_scale_page + h * ld_scale_head
 * + i in k_scale and v_scale (NULL for ECHO_BF16).
 * Constraints: kind one of the three (ECHO_EUNSUP); width a multiple of 8 from
 * 8 to 256, the three ld multiples of 8, page_tokens >= 1, pages and
 * page_tokens < 2^31, heads <= 65535 (ECHO_ESHAPE); k and v 16-byte, the
 * scales 4-byte aligned.
 */
typedef struct echo_cache {
    int64_t pages, page_tokens, heads, width;
    int64_t ld_page, ld_head, ld_token;            /* distances in elements of k and v */
    int64_t ld_scale_page, ld_scale_head;          /* distances in entries of k_scale and v_scale */
    int kind;                                      /* ECHO_BF16, ECHO_I8 or ECHO_I4 */
    void* k;
    void* v;
    void* k_scale;                                 /* float or echo_qparam */
    void* v_scale;
} echo_cache;

/*
 * echo_seqs — the sequences of a call.  `tokens` rows (of new keys and values,
 * of queries, of outputs) belong to `seqs` sequences, one after the other:
 * sequence b has rows starts[b] .. starts[b + 1] - 1, the last ones of its
 * lens[b] tokens.  So row starts[b] + i stands at position
 *   lens[b] - (starts[b + 1] - starts[b]) + i
 * and the token at position t is in slot t % page_tokens of page
 * page_table[b * ld_table + t / page_tokens].
 *
 * These arrays are read on the device and cannot be checked by the host.  The
 * kernels read and write nothing outside the buffers whatever they hold: a
 * token has no place where its position is negative or 2^31 - 2^12 and more, or
 * its entry of the table is past table_pages or names no page.  A sequence whose rows are not all
 * among 0 .. tokens - 1 is not taken; rows of no sequence are left as they were.
 * max_new and max_len (the most rows and the greatest length of a sequence)
 * decide how work is split.  Results are right, but slower, where they are
 * too small or too large; echo_cache_attention may then round otherwise.
 * Constraints: seqs, tokens, table_pages < 2^31, max_new and max_len >= 0
 * (ECHO_ESHAPE); int32 arrays 4-byte aligned.  No sequences or no tokens
 * enqueue nothing.
 */
typedef struct echo_seqs {
    int64_t seqs, tokens, table_pages, ld_table;
    int64_t max_new, max_len;
    const int32_t* starts;                         /* (device) [seqs + 1], from 0, not decreasing */
    const int32_t* lens;                           /* (device) [seqs] */
    const int32_t* page_table;                     /* (device) [seqs][table_pages], rows at ld_table */
} echo_seqs;

/*
 * echo_cache_write — the new tokens' keys and values, quantized on their way
 * into the cache.  Tokens without a place are left out; no two may have the
 * same.  Slots of other tokens are not touched.
 *   k, v (device, in)  [tokens][heads * width], ECHO_F32 or ECHO_BF16 (rounded
 *                      once into an ECHO_BF16 cache), rows at ld_k and ld_v
 * Constraints: tokens * heads <= 2^26 (ECHO_ESHAPE).
 */
int echo_cache_write(const echo_cache* cache, const echo_seqs* seqs, const void* k, int64_t ld_k, const void* v,
                     int64_t ld_v, int dtype, void* stream);

/*
 * echo_cache_read — the same tokens back from the cache as values, (q - z) * s
 * in fp32, rounded once to bf16 where k and v are bf16.  Tokens without a
 * place give NaN.  With starts the sums of lens it reads whole sequences.
 *   k, v (device, out)  [tokens][heads * width], ECHO_F32 or ECHO_BF16
 * Constraints: as for echo_cache_write.
 */
int echo_cache_read(const echo_cache* cache, const echo_seqs* seqs, void* k, int64_t ld_k, void* v, int64_t ld_v,
                    int dtype, void* stream);

/*
 * echo_cache_attention — attention of the new tokens over the cache, in which
 * their own keys and values are already (echo_cache_write):
 *   x_j = scale * sum_d q[d] * k_j[d],  m = max_j x_j,  p_j = exp(x_j - m)
 *   out = sum_j p_j * v_j / sum_j p_j,  lse = m + log sum_j p_j
 * over the tokens j that the row sees: 0 <= j <= position (causal = 1) or
 * 0 <= j < lens (causal = 0), and j > position - window where window > 0.  A
 * row that sees nothing gives 0 and an lse of -infinity.  Query head h reads
 * head h / (q_heads / heads) of the cache.
 * Scores, maxima, sums and outputs are held in fp32.  Products of q with codes
 * are summed before their scale, and v under weights of up to 2^8 (m rises only
 * when a score is that far above it): what leaves fp32 on that way is an
 * infinity.  Products with codes are exact.  For the product with v the weights
 * p_j (times v's scale) are rounded to bf16 or, where the kernel for few query
 * rows takes a sequence, to twice its digits: in calls where max_new (or tokens,
 * if that is less) times q_heads / heads is up to 64, and for sequences of up to
 * 16 such rows in other calls of more than one sequence.  Equal calls give equal
 * bits.
 * A row that sees tokens is NaN, and so is its lse, where q holds an infinity
 * or a NaN, where one of the tokens has no place, and where a score is
 * +infinity or all of them are -infinity.  A score of -infinity beside others,
 * by a key that holds one or by overflow, has the weight 0 that the formulas
 * give it.  Where a key that a row sees holds a NaN, or a value one or an
 * infinity, out is NaN or infinite at least in the elements that the formulas
 * make so, and lse may be NaN with it.  Tokens that a row does not see never
 * touch it.
 *
 *   q (device, in)     bfloat16 bits [tokens][q_heads * width], rows at ld_q
 *   out (device, out)  bfloat16 bits [tokens][q_heads * width], rows at ld_out
 *   lse (device, out)  fp32 [tokens][q_heads], or NULL
 * Constraints: q_heads a multiple of heads, tokens * q_heads <= 2^29, seqs *
 * heads <= 2^22 (ECHO_ESHAPE), scale finite, window >= 0, causal 0 or 1 (ECHO_EINVAL).
 * The workspace (device, 16-byte aligned, at least
 * echo_cache_attention_workspace_bytes of the same arguments) holds what the
 * parts of a long sequence leave to be joined; it may be NULL where that
 * function returns 0.  Calls that may overlap in time need one each.
 */
typedef struct echo_attention_args {
    echo_cache cache;
    echo_seqs seqs;
    int64_t q_heads, ld_q, ld_out;
    int64_t window;                                /* tokens a row sees at most, 0 for all */
    int causal;
    float scale;
    const uint16_t* q;
    uint16_t* out;
    float* lse;
} echo_attention_args;

size_t echo_cache_attention_workspace_bytes(const echo_attention_args* args);
int echo_cache_attention(const echo_attention_args* args, void* workspace, size_t workspace_bytes, void* stream);

/* Static description of a status code. */
const char* echo_status_str(int status);

/* The hipError_t behind the calling thread's last ECHO_EHIP (0 if none). */
int echo_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* ECHO_H */
