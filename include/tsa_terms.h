/*
 * tsa_terms.h -- C ABI of libtsa's attentions with learned score terms, over the schedules and in
 * the manner of tsa.h (types, status codes, the CSR contract, streams, who allocates: see there):
 *
 *   tsa_biased_attention_*        -- a learned bias per head and bucket of the distance q - k;
 *   tsa_differential_attention_*  -- the difference of two softmax maps, weighted by a learned
 *                                    lambda.
 *
 * The pages that tsa.h cites have neither: their scores are scale * q.k alone.
 */
#ifndef TSA_TERMS_H
#define TSA_TERMS_H

#include "tsa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most buckets of a relative position bias. */
#define TSA_MAX_BUCKETS 256

/*
 * Scheduled attention with a learned relative position bias: for query q and key k of lane l,
 * head h = l mod H,
 *   z = scale * <Q[l][q], K[l][k]> + bias[h][b],   b the last bucket with starts[b] <= q - k,
 * and O = softmax(z over the allowed keys) V, with the allowed keys of tsa_scheduled_attention.
 *
 *   Q, K, V       in,  [B*H, S, D] of `dtype`, 16-byte aligned.
 *   row_ptr, col_idx  the CSR of `block`-token blocks; nnz_cap: entries of col_idx.  A row that
 *                 points outside them is empty and reported, as any bad row.
 *   bias          in,  [H, num_buckets] of `dtype` on the device.  A bias of -1e30 or less (the
 *                 lowest bf16 value, -inf) leaves its bucket's keys out.
 *   bucket_starts in,  num_buckets int32 in HOST memory, read during the call: ascending (equal
 *                 starts make an empty bucket), the first one 0; the last bucket is open.
 *   O             out, [B*H, S, D] of `dtype`, 16-byte aligned; rows without keys are 0.
 *   lse           out, [B*H, S] float32, or NULL: the log-sum-exp of z per row, -inf for rows
 *                 without keys; the backward call needs it.
 * Outputs overlap no input and no other output.  Rows of a listed block that the token mask leaves
 * out meet weights of 0 in the products, so they must be finite (padding is zeros, not whatever the
 * memory held); blocks that no row lists are not read.
 *
 * Limits: those of tsa_scheduled_attention, 1 <= num_buckets <= TSA_MAX_BUCKETS,
 * scale >= 1e-30.  Rows past S are neither read nor written, in no lane.  Errors:
 * INVALID_ARGUMENT, UNSUPPORTED, NOT_DEVICE_POINTER, DEVICE_MISMATCH, CUDA; on the device
 * BAD_SCHEDULE (a row is cut at its first bad entry), TIMEOUT.
 */
tsa_status tsa_biased_attention_fwd(const void *Q, const void *K, const void *V,
                                    const int32_t *row_ptr, const int32_t *col_idx, int64_t nnz_cap,
                                    const void *bias, const int32_t *bucket_starts,
                                    int64_t num_buckets, void *O, float *lse, tsa_dtype dtype,
                                    int64_t B, int64_t H, int64_t S, int64_t D, int64_t block,
                                    float scale, tsa_stream_t stream);

/*
 * Differential attention over a schedule: the halves of a head's dimension hold two maps,
 * Q = [q1 | q2] and K = [k1 | k2] of D / 2 each, and
 *   O = (softmax(scale q1.k1) - lambda softmax(scale q2.k2)) V,
 *   lambda = exp(<lambda_q1, lambda_k1>) - exp(<lambda_q2, lambda_k2>) + lambda_init,
 * both maps over the allowed keys of tsa_scheduled_attention, V of the full D.
 *
 *   lambda_q1 .. lambda_k2  in, [lambda_heads, D / 2] of `dtype`; lambda_heads is H (a lambda
 *                 per head) or 1 (one for all).
 *   O             out, [B*H, S, D] of `dtype`, 16-byte aligned; rows without keys are 0.
 *   O2            out, the second map's softmax(..) V, shaped as O, or NULL; the backward call
 *                 needs it.
 *   lse           out, [2, B*H, S] float32: each map's log-sum-exp, or NULL.
 * The maps share their products with K (zeros stand in for the other map's half of Q), so what is not
 * finite in either half of a key makes both maps of the rows that see it NaN; K must be finite, also
 * where an infinity should leave a key out.
 * The other arguments, limits and errors are those of tsa_biased_attention_fwd.
 */
tsa_status tsa_differential_attention_fwd(const void *Q, const void *K, const void *V,
                                          const int32_t *row_ptr, const int32_t *col_idx,
                                          int64_t nnz_cap, const void *lambda_q1,
                                          const void *lambda_k1, const void *lambda_q2,
                                          const void *lambda_k2, int64_t lambda_heads,
                                          float lambda_init, void *O, void *O2, float *lse,
                                          tsa_dtype dtype, int64_t B, int64_t H, int64_t S,
                                          int64_t D, int64_t block, float scale,
                                          tsa_stream_t stream);

/*
 * Backward pass of tsa_biased_attention_fwd: with P the softmax of z over the allowed keys,
 *   Delta = rowsum(dO o O),  dS = P o (dO V^T - Delta),  dV = P^T dO,  dQ = scale dS K,
 *   dK = scale dS^T Q,  dbias[h][b] = sum of dS over the batch's lanes of head h and the pairs
 *   whose distance lies in bucket b,
 * sums in binary32, P and dS rounded to `dtype` for their products (dbias adds dS before its
 * rounding), results rounded once.  (A row of dS sums to zero, so the open last bucket gets
 * minus the sum of the row's others, in rows where any of its own dS is not 0.  It carries
 * their error: Delta's, from the rounded O, times their weights.)  The result does not depend on
 * the order in which thread blocks run.  A gradient beyond the range of `dtype` is an infinity.
 *
 *   O, lse        as the forward call wrote them for the same inputs and CSR.
 *   dO            in,  the upstream gradient, [B*H, S, D] of `dtype`, 16-byte aligned.
 *   dQ, dK, dV    out, [B*H, S, D] of `dtype`, 16-byte aligned.
 *   dbias         out, [H, num_buckets] of `dtype`.
 *   workspace     >= tsa_biased_attention_backward_workspace_bytes(B*H, S, block, nnz_cap,
 *                 num_buckets) bytes, 256-byte aligned; its contents on entry do not matter.
 *                 Calls that may run at the same time, captured graphs among them, need one each.
 * Outputs and workspace overlap no input and one another.  Limits: those of the forward call and
 * of tsa_scheduled_attention_backward (blocks of 64 or 128 tokens, ceil(S/64) <= 8192).  Errors
 * as there.
 */
size_t tsa_biased_attention_backward_workspace_bytes(int64_t lanes, int64_t S, int64_t block,
                                                     int64_t nnz_cap, int64_t num_buckets);
tsa_status tsa_biased_attention_backward(const void *Q, const void *K, const void *V, const void *O,
                                         const void *dO, const float *lse, const int32_t *row_ptr,
                                         const int32_t *col_idx, int64_t nnz_cap, const void *bias,
                                         const int32_t *bucket_starts, int64_t num_buckets,
                                         void *dQ, void *dK, void *dV, void *dbias, tsa_dtype dtype,
                                         int64_t B, int64_t H, int64_t S, int64_t D, int64_t block,
                                         float scale, void *workspace, size_t workspace_bytes,
                                         tsa_stream_t stream);

/*
 * Backward pass of tsa_differential_attention_fwd.  With P1, P2 the two maps' softmax:
 *   dV = (P1 - lambda P2)^T dO,  dS1 = P1 o (dO V^T - rowsum(dO o O1)),
 *   dS2 = -lambda P2 o (dO V^T - rowsum(dO o O2)),  O1 = O + lambda O2,
 *   d[q1 | q2] = scale [dS1 k1 | dS2 k2],  d[k1 | k2] = scale [dS1^T q1 | dS2^T q2],
 *   dlambda = - sum P2 o (dO V^T) over the lanes and rows that share the lambda, and by the chain
 *   rule dlambda_q1 = dlambda exp(<lambda_q1, lambda_k1>) lambda_k1 and so on.
 *
 *   O, O2, lse    as the forward call wrote them for the same inputs and CSR.
 *   dlambda_q1 .. dlambda_k2  out, [lambda_heads, D / 2] of `dtype`.
 *   workspace     >= tsa_differential_attention_backward_workspace_bytes(B*H, S, block, nnz_cap)
 *                 bytes, 256-byte aligned; its contents on entry do not matter.
 * The other arguments, limits and errors are those of tsa_biased_attention_backward.
 */
size_t tsa_differential_attention_backward_workspace_bytes(int64_t lanes, int64_t S, int64_t block,
                                                           int64_t nnz_cap);
tsa_status tsa_differential_attention_backward(
    const void *Q, const void *K, const void *V, const void *O, const void *O2, const void *dO,
    const float *lse, const int32_t *row_ptr, const int32_t *col_idx, int64_t nnz_cap,
    const void *lambda_q1, const void *lambda_k1, const void *lambda_q2, const void *lambda_k2,
    int64_t lambda_heads, float lambda_init, void *dQ, void *dK, void *dV, void *dlambda_q1,
    void *dlambda_k1, void *dlambda_q2, void *dlambda_k2, tsa_dtype dtype, int64_t B, int64_t H,
    int64_t S, int64_t D, int64_t block, float scale, void *workspace, size_t workspace_bytes,
    tsa_stream_t stream);

/*
 * One new token per sequence against a key/value cache: sequence b holds seq_lens[b] tokens, the
 * new one last (its key and value are in the cache already), and its query attends to the keys
 * k < seq_lens[b] of the cache blocks that row b of the schedule lists, with the scores of
 * tsa_biased_attention_fwd (q = seq_lens[b] - 1) or the two maps of
 * tsa_differential_attention_fwd.
 *
 *   Q             in,  [B*H, D] of `dtype`, 16-byte aligned.
 *   K, V          in,  the cache, [B*H, capacity, D] of `dtype`, 16-byte aligned; what it holds at
 *                 and beyond a sequence's length is not read.
 *   seq_lens      in,  [B] int32 on the device, 0 .. capacity.
 *   row_ptr, col_idx  [B + 1] and [nnz_cap] int32 on the device: row b's ascending block indices,
 *                 blocks of `block` tokens of the cache.  Blocks at or beyond the length hold no keys.
 *   O             out, [B*H, D] of `dtype`, 16-byte aligned, overlapping no input; 0 for a sequence
 *                 without keys.
 * One launch, no workspace.  Limits: block in {32, 64, 128}, D in {64, 128}, B*H <= 65535,
 * capacity < 2^31 - 256 (the cache may pass 2^31 elements), scale >= 1e-30.  Errors as the forward
 * calls; on the device BAD_SCHEDULE: a row outside col_idx, a length outside [0, capacity] (the
 * sequence then has no keys), or a block out of order or outside the cache (left out).
 */
tsa_status tsa_biased_attention_decode(const void *Q, const void *K, const void *V,
                                       const int32_t *seq_lens, const int32_t *row_ptr,
                                       const int32_t *col_idx, int64_t nnz_cap, const void *bias,
                                       const int32_t *bucket_starts, int64_t num_buckets, void *O,
                                       tsa_dtype dtype, int64_t B, int64_t H, int64_t capacity,
                                       int64_t D, int64_t block, float scale, tsa_stream_t stream);
tsa_status tsa_differential_attention_decode(
    const void *Q, const void *K, const void *V, const int32_t *seq_lens, const int32_t *row_ptr,
    const int32_t *col_idx, int64_t nnz_cap, const void *lambda_q1, const void *lambda_k1,
    const void *lambda_q2, const void *lambda_k2, int64_t lambda_heads, float lambda_init, void *O,
    tsa_dtype dtype, int64_t B, int64_t H, int64_t capacity, int64_t D, int64_t block, float scale,
    tsa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TSA_TERMS_H */
