/*
 * flashsample_decode.h - C ABI, second part: the LM head in 8-bit integers
 * and beam search. The conventions of flashsample.h hold (device pointers
 * owned by the caller, asynchronous calls on `stream` that allocate nothing
 * and enqueue kernels only, synchronous validation, no mutable global state,
 * no C++ exception across the interface). Every call runs on the calling
 * thread's current device, to which `stream` and all buffers must belong.
 * Calls may run at the same time if none writes what another one uses.
 *
 * The two parts meet in one decode step:
 *
 *   fs_rms_norm_i8   hidden states (+ residual) -> norm -> 8-bit codes + scales
 *   fs_matmul_i8     codes x 8-bit LM head -> logits   (fs_sample_i8: -> tokens)
 *   fs_beam_select   logits + beam scores -> the best continuations
 *   fs_beam_reorder  each beam's cache rows follow the beam it continues
 */
#ifndef FLASHSAMPLE_DECODE_H
#define FLASHSAMPLE_DECODE_H

#include "flashsample.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Rows to 8-bit codes: per row, with a = max |x_j|,
 *     codes[j] = rint(127 x_j / a),   scale = a / 127   (x_j ~ codes[j] scale).
 *   X, ldx, dtype: [M, D] row-major, row stride ldx elements (bf16 or fp32).
 *     X 16-byte aligned, D * sizeof and ldx * sizeof multiples of 16, one row
 *     at most 159 KiB (the row is held on chip).
 *   codes: int8 [M, D], row stride ld_codes >= D, a multiple of 8 (fp32: 4),
 *     and so is the address; an fs_matmul_i8 operand needs both a multiple of 16.
 *   scales: fp32 [M].
 * The codes are those of the exact quotient: ties go to the even code, and no
 * rounding of an intermediate moves one. A row of zeros has codes 0 and scale
 * 0. A row that holds a NaN or an infinity has codes 0 and scale NaN, so what
 * is computed from it is NaN (which never wins in the samplers). */
fs_status_t fs_quantize_i8(const void* X, int64_t ldx, fs_dtype_t dtype, int64_t M, int64_t D, int8_t* codes,
                           int64_t ld_codes, float* scales, hipStream_t stream);

/* Root-mean-square norm with the residual's addition, to 8-bit codes: per row
 *     h = X + residual, rounded to dtype (the sum is formed in fp32),
 *     y_j = h_j gain_j / sqrt(mean(h^2) + eps),
 * and codes, scale of y as in fs_quantize_i8 (exact in the same sense: the
 * norm's factor is common to a row and cancels out of its codes).
 *   residual: null (h = X), or like X, row stride ld_residual.
 *   sum_out: null, or where h goes, row stride ld_sum; needed with a residual,
 *     refused without one. It may be X or residual itself (same address and
 *     stride); other overlaps of buffers are not allowed.
 *   gain: [D] in gain_dtype: dtype or fp32. 16-byte aligned.
 *   eps: >= 0 and finite. */
fs_status_t fs_rms_norm_i8(const void* X, int64_t ldx, const void* residual, int64_t ld_residual, const void* gain,
                           fs_dtype_t gain_dtype, fs_dtype_t dtype, int64_t M, int64_t D, float eps, void* sum_out,
                           int64_t ld_sum, int8_t* codes, int64_t ld_codes, float* scales, hipStream_t stream);

/* 8-bit integer product with a scale per token and per channel:
 *     out[m, n] = round(float(sum_k Q[m, k] W[n, k]) * q_scales[m] * w_scales[n]),
 * the sum exact in 32-bit integers, the two products in fp32 in this order,
 * one rounding to out_dtype.
 *   Q: int8 [M, K], stride ldq; W: int8 [N, K], stride ldw. Both 16-byte
 *     aligned; K, ldq, ldw multiples of 16; K <= 131056 (no sum of products
 *     of 8-bit values can overflow); ldq, ldw < 2^24; M, N <= 2^31 - 2^16.
 *   out: [M, N] in out_dtype (bf16 or fp32), stride ldo >= N, any alignment of
 *     the element type. */
fs_status_t fs_matmul_i8(const int8_t* Q, int64_t ldq, const float* q_scales, const int8_t* W, int64_t ldw,
                         const float* w_scales, int64_t M, int64_t N, int64_t K, void* out, int64_t ldo,
                         fs_dtype_t out_dtype, hipStream_t stream);

/* One token per row from softmax(l / T), l = the fp32 output of fs_matmul_i8
 * on an 8-bit LM head W [V, D]: the product writes the logits to the
 * workspace, the sampler of fs_sample_unfused reads them (same noise, ties,
 * NaN rule and temperature; out_tokens int32 [B]). */
size_t fs_sample_i8_workspace_bytes(int64_t B, int64_t D, int64_t V);
fs_status_t fs_sample_i8(const int8_t* Q, int64_t ldq, const float* q_scales, const int8_t* W, int64_t ldw,
                         const float* w_scales, int64_t B, int64_t D, int64_t V, float temperature, uint64_t seed,
                         uint64_t step, void* workspace, size_t workspace_bytes, int32_t* out_tokens,
                         hipStream_t stream);

/* Beam search's selection. For each of B groups of `beams` rows of logits
 * [B * beams, V] (bf16 or fp32, stride ld_logits, any alignment of the element
 * type) and beam scores [B, beams] (fp32), the n best of the beams * V
 * continuations by
 *     score[b, k] + logits[b, k, v] - log sum exp(logits[b, k, :]),
 * best first, equal ones in order of (k, v). Sums over a row and the scores
 * are kept in fp64 until the end, so their order is not that of rounded
 * scores; equal rows have equal sums whatever their place.
 *   finished: null, or uint8 [B, beams]: a beam whose entry is not zero is not
 *     continued; it stands for itself once, as (k, pad_token, score[b, k]).
 *   n: 1 .. 64; beams: 1 .. 64; V <= 2^31 - 2^15; 0 <= pad_token < V.
 *   out_scores fp32, out_parents (k) and out_tokens (v) int32: [B, n] each.
 *     out_scores may be `scores` itself where n == beams (refused if they
 *     overlap otherwise); no other overlap of buffers is allowed.
 * A beam with score -inf or NaN is not in use; its logits are not read. A
 * logit of -inf never follows; NaN logits are skipped, in the sum too; +inf
 * leaves its beam without continuation. Where fewer than n continuations
 * exist the rest of the outputs are -inf, -1, -1. */
#define FS_BEAM_MAX 64
size_t fs_beam_select_workspace_bytes(int64_t B, int64_t beams, int64_t V, int64_t n, fs_dtype_t logits_dtype);
fs_status_t fs_beam_select(const void* logits, int64_t ld_logits, fs_dtype_t logits_dtype, const float* scores,
                           const uint8_t* finished, int32_t pad_token, int64_t B, int64_t beams, int64_t V, int64_t n,
                           void* workspace, size_t workspace_bytes, float* out_scores, int32_t* out_parents,
                           int32_t* out_tokens, hipStream_t stream);

/* Geometry of one state buffer of beam search, in bytes: `outer` slabs (say
 * layers) of B * beams rows of `blocks` blocks (say heads) of block_bytes
 * contiguous bytes (the positions in use). */
typedef struct fs_beam_layout {
  int64_t outer, outer_stride;
  int64_t row_stride;
  int64_t blocks, block_stride;
  int64_t block_bytes;
} fs_beam_layout_t;

/* Reordering of states: in each of n_states buffers and each slab, row
 * b * beams + i becomes the former row b * beams + parents[b, i]. Rows whose
 * parent is not in 0 .. beams - 1 stay as they are, and so does everything
 * between and behind the blocks.
 *   states: host array of n_states (1 .. 192) device pointers, all of layout
 *     `layout`; out: null (in place: a row that is its own parent is not
 *     touched), or host array of as many device pointers, of layout
 *     `out_layout` (null: `layout`; outer, blocks and block_bytes the same).
 *   parents: device int32 [B, beams]; beams 1 .. 64.
 * block_bytes 0, blocks 0 or outer 0: nothing is done. Refused
 * (FS_ERR_INVALID_ARGUMENT): buffers that overlap, be it with themselves, each
 * other or out; the two arrays are read before the call returns. */
#define FS_BEAM_MAX_STATES 192
fs_status_t fs_beam_reorder(const void* const* states, void* const* out, int64_t n_states,
                            const fs_beam_layout_t* layout, const fs_beam_layout_t* out_layout,
                            const int32_t* parents, int64_t B, int64_t beams, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FLASHSAMPLE_DECODE_H */
