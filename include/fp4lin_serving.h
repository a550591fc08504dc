/*
 * fp4lin_serving.h -- the serving operators of the library: what one step of a
 * served model needs around the 4-bit linear layer.  Part of libfp4lin.so;
 * status codes, conventions (device pointers, streams, host-side checks before
 * any launch, no allocation, no synchronisation) and the tensor-core scale
 * layout are fp4lin.h's.
 *
 *   rmsnorm_mxfp8      RMS norm with the residual's addition and 8-bit output
 *   nvfp4_matvec,      few rows of bf16 or 8-bit activations times 4-bit weights
 *   mxfp4_matvec
 *   kv_block_tables    block tables and slots of a paged cache from request lengths
 *   kv_fp8_store       append to the paged 8-bit cache
 *   kv_fp8_attention   causal attention of new tokens over that cache
 *
 * The 8-bit format ("MXFP8" below): E4M3 elements under one power-of-two scale
 * per block, an E8M0 byte.  For a block whose largest FINITE magnitude is amax,
 * X is the least integer >= -126 with amax <= 448 * 2^X, the byte is X + 127
 * (0 for a block of zeros) and each code is E4M3 round-to-nearest-even of v * 2^-X, so
 * no finite value saturates; infinities saturate to +-448 * 2^X, NaN stays NaN.
 * The value is code * 2^(byte - 127).
 *
 * The paged cache: codes [num_pages, H, P, D] E4M3 bytes and scales
 * [num_pages, H] E8M0 bytes, for K and for V; P rows (tokens) a page, P one of
 * 16, 32, 64, 128; D = 64 or 128.  All P rows of a page and head share a scale.
 * num_pages * P < 2^31.  A slot is page * P + row.
 *
 * The calls of a step (lens: rows in the cache before the step):
 *   kv_block_tables(table, lens, new_lens, ...) -> cu_new, slots
 *   kv_fp8_store(k_new, v_new, slots, ...)
 *   kv_fp8_attention(q, ..., table, lens, cu_new, ...)
 * All of them may be captured into a CUDA graph and replayed.  Each works on
 * its arguments alone: calls on different streams may overlap as long as none
 * writes what another uses (caches, outputs, workspaces).
 */
#ifndef FP4LIN_SERVING_H
#define FP4LIN_SERVING_H

#include "fp4lin.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * s = bf16(x + residual); n = (s / sqrt(mean(s^2) + eps)) * weight; rotated by
 * H_b / sqrt(b) in blocks of b = hadamard along the row when b is 16 or 32
 * (0: not); encoded to MXFP8 with one scale per 32 values.  Sums and the norm
 * are binary32, squares included: |s| below 2^55 and, with eps = 0, rows that
 * reach 2^-55.
 *   x, residual, summed: bf16 [rows, cols], row strides ld_x, ld_r, ld_s
 *     (multiples of 8); residual and summed are both given or both NULL (then
 *     s = x); summed receives s and may be the residual's or x's own memory
 *     with the same row stride, but must not overlap them otherwise;
 *   weight: bf16 [cols]; eps >= 0;
 *   codes: [rows, cols] E4M3 bytes; scales: tensor-core layout of
 *     [rows, cols/32] E8M0 bytes, fp4lin_scale_bytes(rows, cols/32) bytes,
 *     padding written 0; neither overlaps anything else.
 * cols a multiple of 32, at most 32768; pointers 16-byte aligned.
 */
int rmsnorm_mxfp8(const void *x, int64_t ld_x, const void *residual, int64_t ld_r,
                  const void *weight, float eps, int hadamard, int64_t rows, int64_t cols,
                  uint8_t *codes, uint8_t *scales, void *summed, int64_t ld_s, void *stream);

/*
 * y[M, N] = x[M, K] W[N, K]^T with W in the library's 4-bit formats, exactly as
 * nvfp4_quantize / mxfp4_quantize write them, and x in more bits than the W4A4
 * calls take: no activation is rounded to 4 bits.  1 <= M <= 16; there is no
 * form for more rows.  Result bf16_round of a binary32 sum, in a fixed order
 * (the same bits every time), of activations held in f16 under a power of two
 * per row and 256 values.
 *   x_scales NULL: x is bf16 [M, K], row stride ld_x (a multiple of 8);
 *     hadamard = 16 (NVFP4) or 32 (MXFP4) rotates its blocks by H_b / sqrt(b)
 *     on the way in, for weights quantised with that rotation; 0 does not.
 *     Exact down to 2^-31 of the row's largest in 256 values, gone below 2^-39;
 *     rotated values are rounded to f16, 2^-11 of themselves.
 *   x_scales given: x is MXFP8, E4M3 bytes [M, K] with row stride ld_x (a
 *     multiple of 16) and x_scales the tensor-core layout of [M, K/32];
 *     hadamard must be 0 (rmsnorm_mxfp8 rotates what it writes).  Blocks whose
 *     scale is more than 2^21 below the largest of their row in 256 values are
 *     rounded, to 2^-31 of that scale at most.
 *   w_codes [N, K/2]; w_scales tensor-core layout of [N, K/16] (NVFP4) or
 *     [N, K/32] (MXFP4); g_w device float (NVFP4);
 *   y: bf16 [M, N], row stride ldy >= N (any), not overlapping any input.
 * K a multiple of 64, at most 2^24; N any, at most 2^27.  x, x_scales, w_codes,
 * w_scales 16-byte aligned.  MXFP4 blocks whose scale is 2^37 below the largest of
 * their row in 256 values lose bits, from 2^38 on they count as zero.
 */
int nvfp4_matvec(const void *x, const uint8_t *x_scales, int64_t M, int64_t K, int64_t ld_x,
                 int hadamard, const uint8_t *w_codes, const uint8_t *w_scales, const float *g_w,
                 void *y, int64_t N, int64_t ldy, void *stream);
int mxfp4_matvec(const void *x, const uint8_t *x_scales, int64_t M, int64_t K, int64_t ld_x,
                 int hadamard, const uint8_t *w_codes, const uint8_t *w_scales,
                 void *y, int64_t N, int64_t ldy, void *stream);

/*
 * Give B requests the pages that their new tokens need, and say where each new
 * token goes.  Request b holds lens[b] rows and gets new_lens[b] more:
 *   cu_new[b] = new_lens[0] + .. + new_lens[b-1], b = 0 .. B;
 *   with had = ceil(lens/P) and need = ceil((lens + new)/P), the pages
 *   had .. need-1 of table row b are taken from free_pages in order of b,
 *   starting at index *free_head; *next_head is the index behind the last;
 *   slots[cu_new[b] + i] = table[b, p/P] * P + p%P, p = lens[b] + i;
 *   slots from cu_new[B] to max_tokens - 1 are -1.
 * Entries of the table other than those pages are not written.
 *   table [B, width] int32, row stride ld_table; lens, new_lens [B];
 *   free_pages [num_free]; cu_new [B + 1]; slots [max_tokens]; free_head and
 *   next_head one int32 each, not the same one.  Outputs must not overlap
 *   inputs.
 * Recorded as FP4LIN_ERR_OUT_OF_RANGE in the device status word, the rest of
 * the call going on: a negative length (the request gets nothing), rows behind
 * the table's width (no page, slot -1), a free list that runs out (page and
 * slot -1), more than max_tokens new tokens (cu_new stops there), *free_head
 * outside [0, num_free], a negative page in the table where a slot needs it
 * (slot -1).
 * B <= 8192; max_tokens <= 2^30; width * P < 2^31.
 */
int kv_block_tables(int32_t *table, int64_t ld_table, int width, const int32_t *lens,
                    const int32_t *new_lens, int B, const int32_t *free_pages, int num_free,
                    const int32_t *free_head, int page, int max_tokens,
                    int32_t *cu_new, int32_t *slots, int32_t *next_head, void *stream);

/*
 * Append rows to the paged cache: row t of k_new and v_new (bf16 [T, H, D],
 * token strides ld_k, ld_v, multiples of 8) goes to slots[t]; rows of slot -1
 * are skipped.  The new rows of one page must be consecutive tokens with
 * consecutive slots, as kv_block_tables gives them.  Where they begin at the
 * page's row 0, the page starts afresh and its scale is the new rows'; else the
 * page keeps its older rows (0 .. first new row - 1) and takes the larger of
 * its exponent and the new rows', the older rows re-encoded where it grew
 * (exact but for E4M3 subnormals).  Rows behind the last new one are left.
 * A slot outside [-1, num_pages * P) is skipped and recorded as
 * FP4LIN_ERR_OUT_OF_RANGE.  k_new, v_new, k_codes, v_codes 16-byte aligned.
 */
int kv_fp8_store(const void *k_new, int64_t ld_k, const void *v_new, int64_t ld_v,
                 const int32_t *slots, int T, uint8_t *k_codes, uint8_t *k_scales,
                 uint8_t *v_codes, uint8_t *v_scales, int num_pages, int H, int page, int D,
                 void *stream);

/*
 * Causal attention of the step's new tokens over the paged cache (their own
 * rows stored already): with n = cu_new[b+1] - cu_new[b], new token i < n of
 * request b sees positions 0 .. lens[b] + i, found through table row b.  Query
 * head j uses kv head j / G:
 *   o = sum_l softmax(scale * q . k_l) v_l over the visible positions.
 *   q: bf16 [T, H*G, D], token stride ld_q (a multiple of 8), T >= cu_new[B];
 *   out: bf16 [T, H*G, D] contiguous, not overlapping any input; rows of no
 *   request are left as they were;
 *   max_new, max_len: what the host knows of the lengths, n <= max_new and
 *   lens + n <= max_len <= width * P for every request.  A request that breaks
 *   this (or has negative lengths or rows behind T) is skipped, a page outside
 *   [0, num_pages) counts as not visible; both are recorded as
 *   FP4LIN_ERR_OUT_OF_RANGE.  Where cu_new falls anywhere, other requests may be
 *   skipped too.
 * D = 64 or 128; 1 <= G <= 16; B * H <= 65535; max_new * G <= 524280; scale
 * bytes as kv_fp8_store writes them (at most 253).  Rows of the cache behind a
 * request's last may hold anything.  Scores, softmax and sums are binary32.  The
 * softmax weights, each times its page's value scale, are rounded to f16: within
 * 2^-11 of themselves, or 2^-39 of the row's largest (2^-31 where a request has
 * more than 16 (token, head) rows).  Value scales of one request and head are
 * taken to be within 2^64 of one another and at least 2^-80, pages of zeros
 * (byte 0) apart.  workspace: at least
 * kv_fp8_attention_workspace_bytes bytes for the same sizes (may be 0, then
 * NULL will do), 16-byte aligned, of this call alone.
 */
size_t kv_fp8_attention_workspace_bytes(int B, int H, int G, int max_new, int64_t max_len, int D);
int kv_fp8_attention(const void *q, int64_t ld_q, int T, const uint8_t *k_codes,
                     const uint8_t *k_scales, const uint8_t *v_codes, const uint8_t *v_scales,
                     int num_pages, int page, const int32_t *table, int64_t ld_table, int width,
                     const int32_t *lens, const int32_t *cu_new, int max_new, int64_t max_len,
                     float scale, void *out, int B, int H, int G, int D,
                     void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* FP4LIN_SERVING_H */
