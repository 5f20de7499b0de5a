// terms_api.cu -- C entry points of the attentions with learned score terms (include/tsa_terms.h):
// host-side validation, tensor maps and launches.  No call allocates or frees memory.
#include <climits>
#include <cmath>
#include <initializer_list>

#include "tsa_internal.h"
#include "tsa_terms.h"

namespace tsa {
namespace {

// Sizes every form shares.  (A scale of zero or below would turn the masked scores' -inf around.)
tsa_status check_shape(tsa_dtype dtype, int64_t B, int64_t H, int64_t S, int64_t D, int64_t block, float scale,
                       int64_t nnz_cap) {
    if (dtype != TSA_F16 && dtype != TSA_BF16) return TSA_ERR_INVALID_ARGUMENT;
    if (B <= 0 || H <= 0 || S <= 0 || D <= 0 || block <= 0 || nnz_cap < 1) return TSA_ERR_INVALID_ARGUMENT;
    if (!std::isfinite(scale) || scale < 1e-30f) return TSA_ERR_INVALID_ARGUMENT;
    if ((block != 32 && block != 64 && block != 128) || (D != 64 && D != 128)) return TSA_ERR_UNSUPPORTED;
    if (B > 65535 || H > 65535 || B * H > 65535) return TSA_ERR_UNSUPPORTED;
    if (S > INT_MAX || nnz_cap > INT_MAX / 4) return TSA_ERR_UNSUPPORTED;
    return TSA_OK;
}

tsa_status bias_terms(const void *bias, const int32_t *starts, int64_t n, int64_t H, BiasTerms *t) {
    if (!bias || !starts || n < 1) return TSA_ERR_INVALID_ARGUMENT;
    if (n > kMaxBuckets) return TSA_ERR_UNSUPPORTED;
    // the starts are read here, on the host
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, starts) != cudaSuccess) (void)cudaGetLastError();
    else if (at.type == cudaMemoryTypeDevice) return TSA_ERR_INVALID_ARGUMENT;
    if (starts[0] != 0) return TSA_ERR_INVALID_ARGUMENT;
    for (int64_t b = 0; b < n; ++b) {
        if (b > 0 && starts[b] < starts[b - 1]) return TSA_ERR_INVALID_ARGUMENT;
        t->starts[b] = starts[b];
    }
    for (int64_t b = n; b < kMaxBuckets; ++b) t->starts[b] = INT_MAX;
    t->bias = static_cast<const uint16_t *>(bias);
    t->H = (int)H;
    t->n = (int)n;
    return check_aligned({bias}, 1);
}

tsa_status diff_terms(const void *lq1, const void *lk1, const void *lq2, const void *lk2, int64_t heads, float init,
                      int64_t H, int64_t map_rows, DiffTerms *t) {
    if (!lq1 || !lk1 || !lq2 || !lk2) return TSA_ERR_INVALID_ARGUMENT;
    if ((heads != 1 && heads != H) || !std::isfinite(init)) return TSA_ERR_INVALID_ARGUMENT;
    t->lq1 = static_cast<const uint16_t *>(lq1);
    t->lk1 = static_cast<const uint16_t *>(lk1);
    t->lq2 = static_cast<const uint16_t *>(lq2);
    t->lk2 = static_cast<const uint16_t *>(lk2);
    t->H = (int)H;
    t->per_head = heads == H ? 1 : 0;
    t->init = init;
    t->map_rows = map_rows;
    return check_aligned({lq1, lk1, lq2, lk2}, 1);
}

// Maps and launch arguments of a forward call whose arguments have been checked.
struct ForwardMaps {
    CUtensorMap q, k, v, o, o2;
};

tsa_status forward_launch(const void *Q, const void *K, const void *V, const int32_t *row_ptr, const int32_t *col_idx,
                          int64_t nnz_cap, void *O, void *O2, float *lse, tsa_dtype dtype, int64_t lanes, int64_t S,
                          int64_t D, int64_t block, float scale, uint32_t q_rows, tsa_stream_t stream, int dev,
                          ForwardMaps *m, AttnLaunch *a) {
    const bool bf16 = dtype == TSA_BF16;
    const uint64_t L = (uint64_t)lanes, R = (uint64_t)S, C = (uint64_t)D;
    if (!encode_3d(&m->q, Q, bf16, L, R, C, q_rows) || !encode_3d(&m->k, K, bf16, L, R, C, 64) ||
        !encode_3d(&m->v, V, bf16, L, R, C, 64) || !encode_3d(&m->o, O, bf16, L, R, C, 64) ||
        (O2 && !encode_3d(&m->o2, O2, bf16, L, R, C, 64)))
        return TSA_ERR_CUDA;
    a->tmQ = &m->q;
    a->tmK = &m->k;
    a->tmV = &m->v;
    a->tmO = &m->o;
    a->tmO2 = O2 ? &m->o2 : &m->o;
    a->row_ptr = row_ptr;
    a->col_idx = col_idx;
    a->nnz_cap = (int)nnz_cap;
    a->with_o2 = O2 != nullptr;
    a->lse = lse;
    a->nb = (int)((S + 63) / 64);
    a->gran = block == 128 ? 1 : block == 32 ? 2 : 0;
    a->S = (int)S;
    a->D = (int)D;
    a->lanes = (int)lanes;
    a->bf16 = bf16;
    a->scale_log2 = (float)((double)scale * 1.4426950408889634);  // scale * log2(e)
    a->stream = reinterpret_cast<cudaStream_t>(stream);
    return device_flags(dev, &a->flags);
}

// Backward pass: regions of the workspace behind those of the plain pass's layout.  `maps` doubles
// the per-row arrays, `partial` counts the floats of the learned inputs' parts.
struct TermsWorkspace {
    BwdWorkspace plain;
    size_t delta, lse_pad, partial, total;
};

TermsWorkspace terms_workspace(int64_t lanes, int64_t S, int64_t block, int64_t nnz_cap, int64_t maps, int64_t partial) {
    const int64_t nb = (S + 63) / 64, nb_in = block == 128 ? (S + 127) / 128 : 0;
    TermsWorkspace w;
    w.plain = backward_workspace_layout(lanes, S, nb, block == 128 ? 4 * nnz_cap : nnz_cap, nb_in);
    size_t o = w.plain.total;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o = (o + bytes + 255) & ~(size_t)255;
        return at;
    };
    w.delta = w.plain.delta;
    w.lse_pad = w.plain.lse_pad;
    if (maps > 1) {
        w.delta = take(sizeof(float) * (size_t)(maps * lanes * nb * 64));
        w.lse_pad = take(sizeof(float) * (size_t)(maps * lanes * nb * 64));
    }
    w.partial = take(sizeof(float) * (size_t)partial);
    w.total = o;
    return w;
}

tsa_status check_backward_shape(int64_t lanes, int64_t S, int64_t block) {
    if (block != 64 && block != 128) return TSA_ERR_UNSUPPORTED;
    if (lanes * S >= (int64_t)INT_MAX || (S + 63) / 64 > kMaxBackwardBlocks) return TSA_ERR_UNSUPPORTED;
    return TSA_OK;
}

struct BackwardMaps {
    CUtensorMap q, dO, q64, dO64, k, v, dq, dk, dv;
};

tsa_status backward_launch(const void *Q, const void *K, const void *V, const void *O, const void *dO, const float *lse,
                           const int32_t *row_ptr, const int32_t *col_idx, int64_t nnz_cap, void *dQ, void *dK, void *dV,
                           tsa_dtype dtype, int64_t lanes, int64_t S, int64_t D, int64_t block, float scale,
                           uint8_t *w, const TermsWorkspace &ws, tsa_stream_t stream, int dev,
                           BackwardMaps *m, BwdLaunch *a) {
    const bool bf16 = dtype == TSA_BF16;
    const uint64_t L = (uint64_t)lanes, R = (uint64_t)S, C = (uint64_t)D;
    if (!encode_3d(&m->q, Q, bf16, L, R, C, 128) || !encode_3d(&m->dO, dO, bf16, L, R, C, 128) ||
        !encode_3d(&m->q64, Q, bf16, L, R, C, 64) || !encode_3d(&m->dO64, dO, bf16, L, R, C, 64) ||
        !encode_3d(&m->k, K, bf16, L, R, C, 64) || !encode_3d(&m->v, V, bf16, L, R, C, 64) ||
        !encode_3d(&m->dq, dQ, bf16, L, R, C, 64) || !encode_3d(&m->dk, dK, bf16, L, R, C, 64) ||
        !encode_3d(&m->dv, dV, bf16, L, R, C, 64))
        return TSA_ERR_CUDA;
    a->tmQ128 = &m->q;
    a->tmdO128 = &m->dO;
    a->tmQ64 = &m->q64;
    a->tmdO64 = &m->dO64;
    a->tmK64 = &m->k;
    a->tmV64 = &m->v;
    a->tmdQ64 = &m->dq;
    a->tmdK64 = &m->dk;
    a->tmdV64 = &m->dv;
    a->O = static_cast<const uint16_t *>(O);
    a->dO = static_cast<const uint16_t *>(dO);
    a->lse = lse;
    a->row_ptr = row_ptr;
    a->col_idx = col_idx;
    a->nnz_cap = block == 128 ? 4 * nnz_cap : nnz_cap;
    a->read_cap = nnz_cap;
    a->partial = reinterpret_cast<float *>(w + ws.partial);
    a->nb_in = block == 128 ? (int)((S + 127) / 128) : 0;
    a->vlen_in = reinterpret_cast<int *>(w + ws.plain.vlen_in);
    a->rp64 = reinterpret_cast<int32_t *>(w + ws.plain.rp64);
    a->ci64 = reinterpret_cast<int32_t *>(w + ws.plain.ci64);
    a->delta = reinterpret_cast<float *>(w + ws.delta);
    a->lse_pad = reinterpret_cast<float *>(w + ws.lse_pad);
    a->vlen = reinterpret_cast<int *>(w + ws.plain.vlen);
    a->cnt = reinterpret_cast<int *>(w + ws.plain.cnt);
    a->col_ptr = reinterpret_cast<int *>(w + ws.plain.col_ptr);
    a->bitmap = reinterpret_cast<unsigned *>(w + ws.plain.bitmap);
    a->bitmap_bytes = ws.plain.bitmap_bytes;
    a->row_idx = reinterpret_cast<int32_t *>(w + ws.plain.row_idx);
    a->pairs = reinterpret_cast<int *>(w + ws.plain.pairs);
    a->nb = (int)((S + 63) / 64);
    a->S = (int)S;
    a->D = (int)D;
    a->lanes = (int)lanes;
    a->bf16 = bf16;
    a->scale = scale;
    a->stream = reinterpret_cast<cudaStream_t>(stream);
    return device_flags(dev, &a->flags);
}

// The decode calls: everything but the learned inputs.
tsa_status decode_launch(const void *Q, const void *K, const void *V, const int32_t *seq_lens, const int32_t *row_ptr,
                         const int32_t *col_idx, int64_t nnz_cap, void *O, tsa_dtype dtype, int64_t B, int64_t H,
                         int64_t capacity, int64_t D, int64_t block, float scale, tsa_stream_t stream,
                         std::initializer_list<Span> learned, DecodeLaunch *a) {
    if (!Q || !K || !V || !seq_lens || !row_ptr || !col_idx || !O) return TSA_ERR_INVALID_ARGUMENT;
    TSA_TRY(check_shape(dtype, B, H, capacity, D, block, scale, nnz_cap));
    if (capacity > INT_MAX - 256) return TSA_ERR_UNSUPPORTED;
    TSA_TRY(check_aligned({Q, K, V, O}, 15));
    TSA_TRY(check_aligned({seq_lens, row_ptr, col_idx}, 3));
    const int64_t lanes = B * H;
    const size_t one = (size_t)(lanes * D) * 2, cache = one * (size_t)capacity;
    if (outputs_overlap({{O, one}}, {{Q, one}, {K, cache}, {V, cache}, {seq_lens, (size_t)B * 4}, rows_of(row_ptr, B, 1),
                                     entries_of(col_idx, nnz_cap)}))
        return TSA_ERR_INVALID_ARGUMENT;
    for (const Span &s : learned)
        if (overlaps(O, one, s.p, s.bytes)) return TSA_ERR_INVALID_ARGUMENT;
    int dev;
    TSA_TRY(current_device(&dev));
    TSA_TRY(check_device({Q, K, V, seq_lens, row_ptr, col_idx, O}, dev));
    for (const Span &s : learned) TSA_TRY(check_device_ptr(s.p, dev));
    a->Q = static_cast<const uint16_t *>(Q);
    a->K = static_cast<const uint16_t *>(K);
    a->V = static_cast<const uint16_t *>(V);
    a->lens = seq_lens;
    a->row_ptr = row_ptr;
    a->col_idx = col_idx;
    a->nnz_cap = (int)nnz_cap;
    a->O = static_cast<uint16_t *>(O);
    a->lanes = (int)lanes;
    a->H = (int)H;
    a->cap = (int)capacity;
    a->D = (int)D;
    a->block = (int)block;
    TSA_TRY(multiprocessors(dev, &a->sms));
    a->bf16 = dtype == TSA_BF16;
    a->scale_log2 = (float)((double)scale * 1.4426950408889634);
    a->stream = reinterpret_cast<cudaStream_t>(stream);
    return device_flags(dev, &a->flags);
}

// Floats of the tiles' parts, a tile per pair of query blocks: a bias's bucket sums, a lambda's one.
int64_t bias_parts(int64_t lanes, int64_t S, int64_t n) { return lanes * ((S + 127) / 128) * n; }
int64_t lambda_parts(int64_t lanes, int64_t S) { return lanes * ((S + 127) / 128); }

}  // namespace
}  // namespace tsa

using namespace tsa;

extern "C" {

tsa_status tsa_biased_attention_fwd(const void *Q, const void *K, const void *V, const int32_t *row_ptr,
                                    const int32_t *col_idx, int64_t nnz_cap, const void *bias,
                                    const int32_t *bucket_starts, int64_t num_buckets, void *O, float *lse,
                                    tsa_dtype dtype, int64_t B, int64_t H, int64_t S, int64_t D, int64_t block,
                                    float scale, tsa_stream_t stream) {
    if (!Q || !K || !V || !row_ptr || !col_idx || !O) return TSA_ERR_INVALID_ARGUMENT;
    TSA_TRY(check_shape(dtype, B, H, S, D, block, scale, nnz_cap));
    const int64_t lanes = B * H;
    if (lanes * S >= (int64_t)INT_MAX) return TSA_ERR_UNSUPPORTED;
    TSA_TRY(check_aligned({Q, K, V, O}, 15));
    TSA_TRY(check_aligned({row_ptr, col_idx, lse}, 3));
    BiasTerms t;
    TSA_TRY(bias_terms(bias, bucket_starts, num_buckets, H, &t));
    const size_t bytes = (size_t)(lanes * S * D) * 2;
    if (outputs_overlap({{O, bytes}, {lse, (size_t)(lanes * S) * 4}},
                        {{Q, bytes}, {K, bytes}, {V, bytes}, {bias, (size_t)(H * num_buckets) * 2},
                         rows_of(row_ptr, S, block), entries_of(col_idx, nnz_cap)}))
        return TSA_ERR_INVALID_ARGUMENT;
    int dev;
    TSA_TRY(current_device(&dev));
    TSA_TRY(check_device({Q, K, V, row_ptr, col_idx, bias, O, lse}, dev));
    ForwardMaps m;
    AttnLaunch a;
    TSA_TRY(forward_launch(Q, K, V, row_ptr, col_idx, nnz_cap, O, nullptr, lse, dtype, lanes, S, D, block, scale, 128,
                           stream, dev, &m, &a));
    return launch_biased_attention(a, t);
}

tsa_status tsa_differential_attention_fwd(const void *Q, const void *K, const void *V, const int32_t *row_ptr,
                                          const int32_t *col_idx, int64_t nnz_cap, const void *lambda_q1,
                                          const void *lambda_k1, const void *lambda_q2, const void *lambda_k2,
                                          int64_t lambda_heads, float lambda_init, void *O, void *O2, float *lse,
                                          tsa_dtype dtype, int64_t B, int64_t H, int64_t S, int64_t D, int64_t block,
                                          float scale, tsa_stream_t stream) {
    if (!Q || !K || !V || !row_ptr || !col_idx || !O) return TSA_ERR_INVALID_ARGUMENT;
    TSA_TRY(check_shape(dtype, B, H, S, D, block, scale, nnz_cap));
    const int64_t lanes = B * H;
    if (lanes * S >= (int64_t)INT_MAX) return TSA_ERR_UNSUPPORTED;
    TSA_TRY(check_aligned({Q, K, V, O, O2}, 15));
    TSA_TRY(check_aligned({row_ptr, col_idx, lse}, 3));
    DiffTerms t;
    TSA_TRY(diff_terms(lambda_q1, lambda_k1, lambda_q2, lambda_k2, lambda_heads, lambda_init, H, lanes * S, &t));
    const size_t bytes = (size_t)(lanes * S * D) * 2, lb = (size_t)(lambda_heads * D);
    if (outputs_overlap({{O, bytes}, {O2, bytes}, {lse, (size_t)(lanes * S) * 8}},
                        {{Q, bytes}, {K, bytes}, {V, bytes}, {lambda_q1, lb}, {lambda_k1, lb}, {lambda_q2, lb},
                         {lambda_k2, lb}, rows_of(row_ptr, S, block), entries_of(col_idx, nnz_cap)}))
        return TSA_ERR_INVALID_ARGUMENT;
    int dev;
    TSA_TRY(current_device(&dev));
    TSA_TRY(check_device({Q, K, V, row_ptr, col_idx, lambda_q1, lambda_k1, lambda_q2, lambda_k2, O, O2, lse}, dev));
    ForwardMaps m;
    AttnLaunch a;
    TSA_TRY(forward_launch(Q, K, V, row_ptr, col_idx, nnz_cap, O, O2, lse, dtype, lanes, S, D, block, scale, 64, stream,
                           dev, &m, &a));
    return launch_differential_attention(a, t);
}

size_t tsa_biased_attention_backward_workspace_bytes(int64_t lanes, int64_t S, int64_t block, int64_t nnz_cap,
                                                     int64_t num_buckets) {
    if (lanes <= 0 || lanes > 65535 || S <= 0 || S > INT_MAX || nnz_cap < 1 || nnz_cap > INT_MAX / 4) return 0;
    if (check_backward_shape(lanes, S, block) != TSA_OK || num_buckets < 1 || num_buckets > kMaxBuckets) return 0;
    return terms_workspace(lanes, S, block, nnz_cap, 1, bias_parts(lanes, S, num_buckets)).total;
}

tsa_status tsa_biased_attention_backward(const void *Q, const void *K, const void *V, const void *O, const void *dO,
                                         const float *lse, const int32_t *row_ptr, const int32_t *col_idx,
                                         int64_t nnz_cap, const void *bias, const int32_t *bucket_starts,
                                         int64_t num_buckets, void *dQ, void *dK, void *dV, void *dbias,
                                         tsa_dtype dtype, int64_t B, int64_t H, int64_t S, int64_t D, int64_t block,
                                         float scale, void *workspace, size_t workspace_bytes, tsa_stream_t stream) {
    if (!Q || !K || !V || !O || !dO || !lse || !row_ptr || !col_idx || !dQ || !dK || !dV || !dbias || !workspace)
        return TSA_ERR_INVALID_ARGUMENT;
    TSA_TRY(check_shape(dtype, B, H, S, D, block, scale, nnz_cap));
    const int64_t lanes = B * H;
    TSA_TRY(check_backward_shape(lanes, S, block));
    TSA_TRY(check_aligned({Q, K, V, O, dO, dQ, dK, dV}, 15));
    TSA_TRY(check_aligned({lse, row_ptr, col_idx}, 3));
    TSA_TRY(check_aligned({dbias}, 1));
    TSA_TRY(check_aligned({workspace}, 255));
    BiasTerms t;
    TSA_TRY(bias_terms(bias, bucket_starts, num_buckets, H, &t));
    const TermsWorkspace ws = terms_workspace(lanes, S, block, nnz_cap, 1, bias_parts(lanes, S, num_buckets));
    if (workspace_bytes < ws.total) return TSA_ERR_CAPACITY;
    const size_t bytes = (size_t)(lanes * S * D) * 2, bb = (size_t)(H * num_buckets) * 2;
    if (outputs_overlap({{dQ, bytes}, {dK, bytes}, {dV, bytes}, {dbias, bb}, {workspace, ws.total}},
                        {{Q, bytes}, {K, bytes}, {V, bytes}, {O, bytes}, {dO, bytes}, {lse, (size_t)(lanes * S) * 4},
                         {bias, bb}, rows_of(row_ptr, S, block), entries_of(col_idx, nnz_cap)}))
        return TSA_ERR_INVALID_ARGUMENT;
    int dev;
    TSA_TRY(current_device(&dev));
    TSA_TRY(check_device({Q, K, V, O, dO, lse, row_ptr, col_idx, bias, dQ, dK, dV, dbias, workspace}, dev));
    BackwardMaps m;
    BwdLaunch a;
    TSA_TRY(backward_launch(Q, K, V, O, dO, lse, row_ptr, col_idx, nnz_cap, dQ, dK, dV, dtype, lanes, S, D, block,
                            scale, static_cast<uint8_t *>(workspace), ws, stream, dev, &m, &a));
    return launch_biased_backward(a, t, static_cast<uint16_t *>(dbias));
}

size_t tsa_differential_attention_backward_workspace_bytes(int64_t lanes, int64_t S, int64_t block, int64_t nnz_cap) {
    if (lanes <= 0 || lanes > 65535 || S <= 0 || S > INT_MAX || nnz_cap < 1 || nnz_cap > INT_MAX / 4) return 0;
    if (check_backward_shape(lanes, S, block) != TSA_OK) return 0;
    return terms_workspace(lanes, S, block, nnz_cap, 2, lambda_parts(lanes, S)).total;
}

tsa_status tsa_differential_attention_backward(const void *Q, const void *K, const void *V, const void *O,
                                               const void *O2, const void *dO, const float *lse,
                                               const int32_t *row_ptr, const int32_t *col_idx, int64_t nnz_cap,
                                               const void *lambda_q1, const void *lambda_k1, const void *lambda_q2,
                                               const void *lambda_k2, int64_t lambda_heads, float lambda_init,
                                               void *dQ, void *dK, void *dV, void *dlambda_q1, void *dlambda_k1,
                                               void *dlambda_q2, void *dlambda_k2, tsa_dtype dtype, int64_t B,
                                               int64_t H, int64_t S, int64_t D, int64_t block, float scale,
                                               void *workspace, size_t workspace_bytes, tsa_stream_t stream) {
    if (!Q || !K || !V || !O || !O2 || !dO || !lse || !row_ptr || !col_idx || !dQ || !dK || !dV || !dlambda_q1 ||
        !dlambda_k1 || !dlambda_q2 || !dlambda_k2 || !workspace)
        return TSA_ERR_INVALID_ARGUMENT;
    TSA_TRY(check_shape(dtype, B, H, S, D, block, scale, nnz_cap));
    const int64_t lanes = B * H;
    TSA_TRY(check_backward_shape(lanes, S, block));
    TSA_TRY(check_aligned({Q, K, V, O, O2, dO, dQ, dK, dV}, 15));
    TSA_TRY(check_aligned({lse, row_ptr, col_idx}, 3));
    TSA_TRY(check_aligned({dlambda_q1, dlambda_k1, dlambda_q2, dlambda_k2}, 1));
    TSA_TRY(check_aligned({workspace}, 255));
    DiffTerms t;
    // the per-row arrays are the workspace's, padded to whole blocks
    TSA_TRY(diff_terms(lambda_q1, lambda_k1, lambda_q2, lambda_k2, lambda_heads, lambda_init, H,
                       lanes * ((S + 63) / 64) * 64, &t));
    const TermsWorkspace ws = terms_workspace(lanes, S, block, nnz_cap, 2, lambda_parts(lanes, S));
    if (workspace_bytes < ws.total) return TSA_ERR_CAPACITY;
    const size_t bytes = (size_t)(lanes * S * D) * 2, lb = (size_t)(lambda_heads * D);
    if (outputs_overlap({{dQ, bytes}, {dK, bytes}, {dV, bytes}, {dlambda_q1, lb}, {dlambda_k1, lb}, {dlambda_q2, lb},
                         {dlambda_k2, lb}, {workspace, ws.total}},
                        {{Q, bytes}, {K, bytes}, {V, bytes}, {O, bytes}, {O2, bytes}, {dO, bytes},
                         {lse, (size_t)(lanes * S) * 8}, {lambda_q1, lb}, {lambda_k1, lb}, {lambda_q2, lb},
                         {lambda_k2, lb}, rows_of(row_ptr, S, block), entries_of(col_idx, nnz_cap)}))
        return TSA_ERR_INVALID_ARGUMENT;
    int dev;
    TSA_TRY(current_device(&dev));
    TSA_TRY(check_device({Q, K, V, O, O2, dO, lse, row_ptr, col_idx, lambda_q1, lambda_k1, lambda_q2, lambda_k2, dQ, dK,
                          dV, dlambda_q1, dlambda_k1, dlambda_q2, dlambda_k2, workspace}, dev));
    BackwardMaps m;
    BwdLaunch a;
    TSA_TRY(backward_launch(Q, K, V, O, dO, lse, row_ptr, col_idx, nnz_cap, dQ, dK, dV, dtype, lanes, S, D, block,
                            scale, static_cast<uint8_t *>(workspace), ws, stream, dev, &m, &a));
    uint16_t *const dl[4] = {static_cast<uint16_t *>(dlambda_q1), static_cast<uint16_t *>(dlambda_k1),
                             static_cast<uint16_t *>(dlambda_q2), static_cast<uint16_t *>(dlambda_k2)};
    return launch_differential_backward(a, t, static_cast<const uint16_t *>(O2), dl);
}

tsa_status tsa_biased_attention_decode(const void *Q, const void *K, const void *V, const int32_t *seq_lens,
                                       const int32_t *row_ptr, const int32_t *col_idx, int64_t nnz_cap,
                                       const void *bias, const int32_t *bucket_starts, int64_t num_buckets, void *O,
                                       tsa_dtype dtype, int64_t B, int64_t H, int64_t capacity, int64_t D,
                                       int64_t block, float scale, tsa_stream_t stream) {
    BiasTerms t;
    if (H <= 0 || H > 65535) return H <= 0 ? TSA_ERR_INVALID_ARGUMENT : TSA_ERR_UNSUPPORTED;
    TSA_TRY(bias_terms(bias, bucket_starts, num_buckets, H, &t));
    DecodeLaunch a;
    TSA_TRY(decode_launch(Q, K, V, seq_lens, row_ptr, col_idx, nnz_cap, O, dtype, B, H, capacity, D, block, scale, stream,
                          {{bias, (size_t)(H * num_buckets) * 2}}, &a));
    return launch_biased_decode(a, t);
}

tsa_status tsa_differential_attention_decode(const void *Q, const void *K, const void *V, const int32_t *seq_lens,
                                             const int32_t *row_ptr, const int32_t *col_idx, int64_t nnz_cap,
                                             const void *lambda_q1, const void *lambda_k1, const void *lambda_q2,
                                             const void *lambda_k2, int64_t lambda_heads, float lambda_init, void *O,
                                             tsa_dtype dtype, int64_t B, int64_t H, int64_t capacity, int64_t D,
                                             int64_t block, float scale, tsa_stream_t stream) {
    DiffTerms t;
    if (H <= 0 || H > 65535) return H <= 0 ? TSA_ERR_INVALID_ARGUMENT : TSA_ERR_UNSUPPORTED;
    if (D != 64 && D != 128) return D <= 0 ? TSA_ERR_INVALID_ARGUMENT : TSA_ERR_UNSUPPORTED;
    TSA_TRY(diff_terms(lambda_q1, lambda_k1, lambda_q2, lambda_k2, lambda_heads, lambda_init, H, 0, &t));
    const size_t lb = (size_t)(lambda_heads * D);
    DecodeLaunch a;
    TSA_TRY(decode_launch(Q, K, V, seq_lens, row_ptr, col_idx, nnz_cap, O, dtype, B, H, capacity, D, block, scale, stream,
                          {{lambda_q1, lb}, {lambda_k1, lb}, {lambda_q2, lb}, {lambda_k2, lb}}, &a));
    return launch_differential_decode(a, t);
}

}  // extern "C"
