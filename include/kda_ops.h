/*
 * kda_ops.h -- C ABI of libkda.so, continued: the operators a layer runs
 * around and beside the KDA core of kda.h (whose return codes, error bits,
 * state-pool layout and stream rules they share).
 *
 *   kda_quant_rows   residual addition, RMSNorm and int8 rows with one scale each
 *   kda_linear_i8    y = x . W^T on int8 operands with row and column scales
 *   kda_la_step      linear attention with a decay a head, one token a sequence
 *   kda_la_prefill   the same attention over packed prompts
 *
 * kda_quant_rows -> kda_linear_i8 is the 8-bit form of the projections
 * (kda_linear) in front of and after the core; kda_la_prefill leaves the
 * states that kda_la_step continues from, in the pool layout of kda_step.
 *
 * All pointers are DEVICE pointers on the current device; the caller keeps
 * them alive until the call has completed on its stream.  Calls are
 * asynchronous, take no host sync and can be captured into a CUDA graph.  They
 * keep no state between calls, so any host thread may make them.
 * Kernels may be set up while the stream's work before them still runs (dependent launches); they
 * touch global memory only when it has ended.
 */
#ifndef KDA_OPS_H
#define KDA_OPS_H

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/* kda_la_check: cu_seqlens of a sequence out of order or range, or longer than
 * max_len: the sequence is skipped. */
#define KDA_ERR_SEQ 16u

/* Columns of a row that kda_quant_rows takes at most. */
#define KDA_QUANT_MAX_COLS 32768

/*
 * kda_quant_rows -- int8 rows with one fp32 scale each, from bf16 rows:
 *     h = x + residual, rounded to bf16 and written back to residual
 *         (residual NULL: h = x, nothing written);
 *     p = h * norm_weight, n = 1 / sqrt(mean(h^2) + eps)
 *         (norm_weight NULL: p = h, n = 1);
 *     q = round(127 p / max|p|), ties to even, in -127..127
 *     scale = n max|p| / 127
 * so that q * scale is the RMSNorm of h (or h itself) quantised once, with no
 * rounding to bf16 in between.  The norm's factor n cancels in q, and the
 * kernel decides each q exactly.  A row of zeros has q = 0 and scale 0; a row
 * with a NaN or an infinity in p has q = 0 and scale NaN, which a product with
 * the row then shows.
 *
 *   x            bf16 [rows, cols], row stride ldx           (read)
 *   residual     bf16 [rows, cols], row stride ldr, or NULL  (read, written)
 *   norm_weight  bf16 [cols], or NULL
 *   eps          >= 0 (read only with norm_weight)
 *   q            int8 [rows, cols], row stride ldq           (written)
 *   scales       fp32 [rows]                                 (written)
 * cols a multiple of 16 up to KDA_QUANT_MAX_COLS; x, residual and norm_weight
 * 16-byte aligned, ldx and ldr multiples of 8; q 8-byte aligned, ldq a
 * multiple of 8; scales 4-byte aligned.  residual may be x itself; q and
 * scales overlap none of the others.  rows = 0 enqueues nothing.  Returns
 * KDA_OK, KDA_EINVAL or KDA_ECUDA.
 */
int kda_quant_rows(const void* x, long long rows, long long ldx, long long cols, void* residual, long long ldr,
                   const void* norm_weight, float eps, void* q, long long ldq, float* scales, void* cuda_stream);

/*
 * kda_linear_i8 -- y[m, n] = x_scales[m] w_scales[n] sum_k x[m, k] W[n, k], rounded once
 * to bf16: the product of int8 rows (kda_quant_rows: one scale a token) with
 * an int8 weight that has one scale an output channel.
 *
 *   x, x_scales  int8 [rows, K] (row stride ldx), fp32 [rows]
 *   w, w_scales  int8 [N, K] row-major (a torch Linear weight), fp32 [N]
 *   y            bf16 [rows, N], row stride ldy               (written)
 * K a multiple of 16; x and W 16-byte aligned with ldx % 16 == 0, y 2-byte
 * and the scales 4-byte aligned; y overlaps none of the inputs.  Every int8
 * value is allowed, -128 too.  The sum is exact while the partial sums stay
 * below 2^24 and is rounded to fp32 beyond.  rows = 0 enqueues nothing.
 * Returns KDA_OK, KDA_EINVAL or KDA_ECUDA.
 */
int kda_linear_i8(const void* x, long long rows, long long ldx, const float* x_scales, const void* w,
                  const float* w_scales, long long N, long long K, void* y, long long ldy, void* cuda_stream);

/*
 * kda_linear_i8_check -- as kda_linear_check, for kda_linear_i8: synchronise
 * `cuda_stream`, read and clear the device error bits (KDA_ERR_TIMEOUT: a
 * launch gave up waiting for its own copies; its y is not meaningful).
 */
int kda_linear_i8_check(void* cuda_stream, unsigned* device_flags);

/*
 * Linear attention with a decay a head.  For value head h (of `heads`) and its
 * query / key head h / (heads / qk_heads), a state S [128 (v), 128 (k)] and a
 * log decay g <= 0:
 *     S_t = exp(g_t) S_{t-1} + v_t k_t^T        o_t = scale S_t q_t
 * States live in the pool of kda_step: [pool, heads, 128 (v), 128 (k)], fp32
 * or bf16 (KDA_STATE_F32 / KDA_STATE_BF16; computed in fp32, the stored state
 * rounded), indexed by slots.
 *
 *   q, k         bf16 [rows, qk_heads, 128], row strides ldq, ldk
 *   v, out       bf16 [rows, heads, 128], row strides ldv, ldo
 *   g            fp32: ldg = 0: [heads], one decay a head for every token;
 *                else [rows, heads] with row stride ldg >= heads.  -inf drops the state.
 *   state_pool   [pool_slots, heads, 128, 128], 16-byte aligned (read, written)
 * heads 1..65535, a multiple of qk_heads; q, k, v 16-byte aligned with row
 * strides that are multiples of 8, out 16-byte aligned with ldo % 8 == 0.  The
 * inputs may be columns of one packed projection row.  out overlaps none of
 * them.
 */

/*
 * kda_la_step -- one token for each of `rows` sequences: row b reads and
 * writes the state of slots[b] (int32 [rows]).  slots[b] = -1 is a padding
 * row: no state is touched and its out row is zero; any other slot outside
 * [0, pool_slots) sets KDA_ERR_SLOT and the row is skipped.  The same slot
 * twice in one call is undefined behaviour.  rows = 0 enqueues nothing.
 * Returns KDA_OK, KDA_EINVAL or KDA_ECUDA.
 */
int kda_la_step(const void* q, long long ldq, const void* k, long long ldk, const void* v, long long ldv,
                long long rows, int heads, int qk_heads, const float* g, long long ldg, float scale,
                void* state_pool, int state_dtype, long long pool_slots, const int* slots, void* out, long long ldo,
                void* cuda_stream);

/*
 * kda_la_prefill -- the tokens of `seqs` sequences, packed one after the other:
 * sequence i has the rows cu_seqlens[i] .. cu_seqlens[i + 1] - 1 and leaves the state
 * behind its last token in slots[i].
 *
 *   cu_seqlens   int32 [seqs + 1], ascending, in 0..rows
 *   max_len      at least the longest sequence's length (a larger value costs only time)
 *   has_state    int32 [seqs], nonzero: the sequence continues from the state in slots[i];
 *                or NULL: every sequence starts from zeros
 *   slots        int32 [seqs]; -1 is a padding sequence (its out rows zero, no state
 *                touched); a bad slot sets KDA_ERR_SLOT, a bad pair of cu_seqlens or a
 *                length above max_len KDA_ERR_SEQ, and the sequence is skipped
 *   workspace    kda_la_prefill_workspace(...) bytes of device memory, 16-byte aligned (NULL
 *                if that is 0).  Calls that may run at the same time need one each.
 * A sequence without tokens keeps its state, or, without has_state, gets a state of zeros.
 * Rows behind the last sequence are left as they are.  rows up to 2^31 - 1;
 * seqs = 0 enqueues nothing.  Returns KDA_OK, KDA_EINVAL or KDA_ECUDA.
 */
int kda_la_prefill(const void* q, long long ldq, const void* k, long long ldk, const void* v, long long ldv,
                   long long rows, int heads, int qk_heads, const float* g, long long ldg, float scale,
                   const int* cu_seqlens, long long seqs, long long max_len, const int* has_state,
                   void* state_pool, int state_dtype, long long pool_slots, const int* slots, void* out,
                   long long ldo, void* workspace, long long workspace_bytes, void* cuda_stream);

/* kda_la_prefill_workspace -- the bytes of workspace that a kda_la_prefill of these sizes
 * takes on the current device (0 too where the sizes are invalid). */
long long kda_la_prefill_workspace(long long rows, int heads, long long seqs, long long max_len);

/*
 * kda_la_check -- synchronise `cuda_stream`, then read and clear the device error bits
 * (KDA_ERR_SLOT, KDA_ERR_SEQ, KDA_ERR_TIMEOUT) that kda_la_step and kda_la_prefill have set
 * on the current device.  Returns KDA_OK, KDA_EINVAL (device_flags NULL) or KDA_ECUDA.
 */
int kda_la_check(void* cuda_stream, unsigned* device_flags);

#ifdef __cplusplus
}
#endif

#endif /* KDA_OPS_H */
