/*
 * tsa_cache.h -- C ABI of libtsa's rotary positions, paged key/value cache and the plain attention's
 * one-token form over it, in the manner of tsa.h (types, status codes, the CSR contract, streams, who
 * allocates: see there):
 *
 *   tsa_rotary                  -- rotates the pairs of Q's and K's rows by their positions (and back);
 *   tsa_paged_append            -- writes new tokens to a paged cache, rotating on the way;
 *   tsa_paged_attention_decode  -- one new token per sequence against a paged cache.
 *
 * The pages that tsa.h cites have none of them: their rows carry no positions, and they serve no tokens.
 *
 * A paged cache is two arrays K_cache, V_cache of num_pages pages; a page holds page_size tokens of every
 * key/value head, [HK, page_size, D] contiguous, and page p begins p * page_stride elements into its array
 * (page_stride >= HK * page_size * D, any for one page: both arrays may be slices of one).  page_table[b][i] is the page of
 * sequence b's tokens [i * page_size, (i + 1) * page_size); what entries that no token reaches hold does not matter.
 *
 * Rows of Q, K, V and of the rotated outputs are D contiguous elements; `strides` (int64 in HOST memory,
 * read during the call) gives, for each tensor in the order stated, the elements from one batch, head and
 * token to the next: not negative, multiples of 8 (along an axis of one, any).  NULL: all are contiguous
 * [B, heads, tokens, D].
 */
#ifndef TSA_CACHE_H
#define TSA_CACHE_H

#include "tsa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest row that is rotated or appended. */
#define TSA_MAX_ROTARY_DIM 256

/*
 * Rotary positions: with p the row's position and f_i = frequencies[i], i < R / 2, R = rotary_dim, the pair
 * (x_j, x_k) of every row of Q and K becomes
 *   magnitude * (x_j cos(p f_i) - x_k sin(p f_i),  x_k cos(p f_i) + x_j sin(p f_i)),
 * (j, k) = (i, i + R / 2), or (2 i, 2 i + 1) if `interleaved`; dimensions from R on are copied.  `inverse`
 * rotates by -p f_i: with the upstream gradients for Q and K it is the backward pass.
 *
 *   Q             in,  [B, H, S, D] of `dtype`, 16-byte aligned.
 *   K             in,  [B, HK, S, D] of `dtype`, 16-byte aligned, or NULL (then K_out too; HK is not read).
 *   strides       12 values: Q, K, Q_out, K_out.
 *   positions     in,  [position_rows, S] int32 on the device, position_rows 1 (all sequences') or B; any
 *                 value, negative ones too.  NULL: 0 .. S - 1.
 *   frequencies   in,  R / 2 binary64 in HOST memory, read during the call: finite, |f| <= 65536.
 *   Q_out, K_out  out, shaped as Q and K.  They may be Q and K themselves, with the same strides;
 *                 otherwise outputs share no memory with an input or one another.  Tensors whose rows lie in
 *                 one another's gaps, as parts of a joint projection do ([B, S, H + 2 HK, D], [B, S, H, 3, D],
 *                 [B, H + 2 HK, S, D]), share none; they need the same strides, a batch's a multiple of a
 *                 token's or the reverse.
 * Angles are kept as 64-bit fractions of a turn: |p| 2^-65 turns off at most, whatever the position;
 * products and sums are binary32, results rounded once.
 *
 * Limits: D a multiple of 16 up to TSA_MAX_ROTARY_DIM, R a multiple of 16 up to D, B * S < 2^31,
 * H, HK <= 65535.  Errors: INVALID_ARGUMENT, UNSUPPORTED, NOT_DEVICE_POINTER, DEVICE_MISMATCH, CUDA.
 */
tsa_status tsa_rotary(const void *Q, const void *K, const int64_t *strides, const int32_t *positions,
                      int64_t position_rows, const double *frequencies, int64_t rotary_dim,
                      int interleaved, float magnitude, int inverse, void *Q_out, void *K_out,
                      tsa_dtype dtype, int64_t B, int64_t H, int64_t HK, int64_t S, int64_t D,
                      tsa_stream_t stream);

/*
 * New tokens to a paged cache: sequence b holds seq_lens[b] tokens with its counts[b] new ones, which are
 * its last.  Token t < counts[b] of K, V (and Q) has position p = seq_lens[b] - counts[b] + t; K's row,
 * rotated as by tsa_rotary, and V's are written to slot p % page_size of page page_table[b][p / page_size],
 * and Q's row is rotated into Q_out.  Rows t >= counts[b] and rows of negative positions (a batch padded in
 * front) are no tokens: their Q_out is 0, and nothing is written for them to the cache, which keeps what it
 * holds everywhere else.
 *
 *   Q             in,  [B, H, T, D] of `dtype`, 16-byte aligned, or NULL (then Q_out too; H is not read).
 *   K, V          in,  [B, HK, T, D] of `dtype`, 16-byte aligned.
 *   strides       12 values: Q, K, V, Q_out.
 *   K_cache, V_cache  in/out, 16-byte aligned, page strides multiples of 8.
 *   page_table    in,  [B, max_pages] int32 on the device.
 *   seq_lens      in,  [B] int32 on the device, 0 .. max_pages * page_size.
 *   counts        in,  [B] int32 on the device, 0 .. T, or NULL: T each.
 *   frequencies   as for tsa_rotary, or NULL: K is written as it is (then Q must be NULL).
 *   Q_out         out, shaped as Q; Q itself, with the same strides, or sharing no memory with an input.
 * The slots written must be distinct: no two sequences may write to one page's slot.  The caches share no
 * memory with one another or with an input.
 *
 * Limits: those of tsa_rotary, page_size in {16, 32, 64, 128, 256}, num_pages < 2^31, max_pages * page_size <
 * 2^31 - 256, B * T < 2^31 (the cache may pass 2^31 elements).  Errors as for tsa_rotary; on the device
 * BAD_SCHEDULE: a length or a count out of its range (the sequence then has no tokens), or a token's page
 * outside the cache (its K and V are left out).
 */
tsa_status tsa_paged_append(const void *Q, const void *K, const void *V, const int64_t *strides,
                            void *K_cache, void *V_cache, int64_t num_pages, int64_t page_size,
                            int64_t k_page_stride, int64_t v_page_stride, const int32_t *page_table,
                            int64_t max_pages, const int32_t *seq_lens, const int32_t *counts,
                            const double *frequencies, int64_t rotary_dim, int interleaved,
                            float magnitude, void *Q_out, tsa_dtype dtype, int64_t B, int64_t H,
                            int64_t HK, int64_t T, int64_t D, tsa_stream_t stream);

/*
 * One new token per sequence against a paged cache: sequence b holds seq_lens[b] tokens, the new one last
 * (its key and value are in the cache already), and O = softmax(scale q.k) V over its keys, or over those
 * of the key blocks that row b of a schedule lists.  Query head h reads key/value head h / (H / HK).
 *
 *   Q             in,  [B, H, D] of `dtype`, 16-byte aligned.
 *   K_cache, V_cache  in, 16-byte aligned, page strides multiples of 8; slots of no token are not read.
 *   page_table    in,  [B, max_pages] int32 on the device.
 *   seq_lens      in,  [B] int32 on the device, 0 .. max_pages * page_size.
 *   row_ptr, col_idx  [B + 1] and [nnz_cap] int32 on the device: row b's ascending block indices, blocks of
 *                 `block` tokens of the sequence (of any size beside the page's); blocks at or beyond the
 *                 length hold no keys.  Both NULL (nnz_cap 0): every key.
 *   O             out, [B, H, D] of `dtype`, 16-byte aligned, overlapping no input; 0 for a sequence
 *                 without keys.
 *   workspace     >= tsa_paged_attention_decode_workspace_bytes(..) bytes, 256-byte aligned, or NULL where
 *                 that is 0; its contents on entry do not matter.  Calls that may run at the same time,
 *                 captured graphs among them, need one each.
 * Scores, weights and sums are binary32; a weight meets V as a sum of numbers of `dtype`, in bf16 all of it, in f16
 * all but 2^-22 of it or 2^-39 of the row's largest.  The result does not depend on the order in which thread blocks
 * run.  A NaN or +inf score makes the row NaN; V must be finite in every key that is listed, also where a score of
 * -inf leaves the key without weight.
 *
 * Limits: block in {32, 64, 128}, D in {64, 128}, H a multiple of HK, B * H <= 65535, page sizes and tables as
 * for tsa_paged_append, scale >= 1e-30.  Errors: those of tsa_paged_append and CAPACITY; on the device
 * BAD_SCHEDULE: a length out of its range or a row outside col_idx (the sequence then has no keys), a block
 * out of order or outside the sequence's pages or a page outside the cache (its keys are left out).
 */
size_t tsa_paged_attention_decode_workspace_bytes(int64_t B, int64_t H, int64_t HK, int64_t D,
                                                  int64_t page_size, int64_t max_pages, int64_t block,
                                                  int64_t nnz_cap);
tsa_status tsa_paged_attention_decode(const void *Q, const void *K_cache, const void *V_cache,
                                      int64_t num_pages, int64_t page_size, int64_t k_page_stride,
                                      int64_t v_page_stride, const int32_t *page_table,
                                      int64_t max_pages, const int32_t *seq_lens,
                                      const int32_t *row_ptr, const int32_t *col_idx, int64_t nnz_cap,
                                      void *O, tsa_dtype dtype, int64_t B, int64_t H, int64_t HK,
                                      int64_t D, int64_t block, float scale, void *workspace,
                                      size_t workspace_bytes, tsa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TSA_CACHE_H */
