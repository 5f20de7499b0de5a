// terms_api.cu -- C entry points of the attentions with learned score terms (include/tsa.h):
// host-side validation, tensor maps and launches.  No call allocates or frees memory.
#include <climits>
#include <cmath>
#include <initializer_list>

#include "tsa_internal.h"

namespace tsa {
namespace {

struct Span {
    const void *p;
    size_t bytes;
};

// No output may overlap an input or another output.
bool outputs_overlap(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (const Span *o = outs.begin(); o != outs.end(); ++o) {
        if (!o->p) continue;
        for (const Span &i : ins)
            if (i.p && overlaps(o->p, o->bytes, i.p, i.bytes)) return true;
        for (const Span *q = o + 1; q != outs.end(); ++q)
            if (q->p && overlaps(o->p, o->bytes, q->p, q->bytes)) return true;
    }
    return false;
}

tsa_status check_aligned(std::initializer_list<const void *> ptrs, uintptr_t mask) {
    for (const void *p : ptrs)
        if (p && (reinterpret_cast<uintptr_t>(p) & mask)) return TSA_ERR_INVALID_ARGUMENT;
    return TSA_OK;
}

tsa_status check_device(std::initializer_list<const void *> ptrs, int dev) {
    for (const void *p : ptrs)
        if (p) TSA_TRY(check_device_ptr(p, dev));
    return TSA_OK;
}

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
    a->O = static_cast<uint16_t *>(O2);
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
                        {{Q, bytes}, {K, bytes}, {V, bytes}, {bias, (size_t)(H * num_buckets) * 2}}))
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
                         {lambda_k2, lb}}))
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

}  // extern "C"
