// cache_api.cu -- C entry points of the rotary positions, the paged cache and its one-token attention
// (include/tsa_cache.h): host-side validation and launches.  No call allocates or frees memory.
#include <algorithm>
#include <climits>
#include <cmath>

#include "tsa_cache.h"
#include "tsa_internal.h"

namespace tsa {
namespace {

static_assert(kMaxRotaryDim == TSA_MAX_ROTARY_DIM, "the header's limit");

// Memory of rows: `inner` contiguous elements repeated over strided axes (batch, head and token; a cache's pages).
struct Field {
    const void *p = nullptr;
    int64_t n[3] = {1, 1, 1}, stride[3] = {0, 0, 0}, inner = 0;  // elements of 2 bytes
};

constexpr int64_t kMaxExtent = int64_t{1} << 58;  // elements: no sum of offsets below overflows

bool extent(const Field &f, int64_t *elements) {
    __int128 e = f.inner;
    for (int i = 0; i < 3; ++i) e += (__int128)(f.n[i] - 1) * f.stride[i];
    *elements = (int64_t)e;
    return e <= kMaxExtent;
}

Span span_of(const Field &f) {
    int64_t e = 0;
    (void)extent(f, &e);
    return {f.p, (size_t)e * 2};
}

// Two fields that repeat with the same strides, largest first.
struct Pair {
    int64_t na[3], nb[3], stride[3], inner_a, inner_b;

    // Whether rows of the axes from `axis` on meet, b's `delta` elements behind a's.  The axis's steps count only as far
    // as what is left of a and b reaches: two where one of the fields does not overlap itself.  (More are not looked
    // into, and taken to meet.)
    bool meet(int axis, int64_t delta) const {
        int64_t ea = inner_a, eb = inner_b;
        for (int i = axis; i < 3; ++i) {
            ea += (na[i] - 1) * stride[i];
            eb += (nb[i] - 1) * stride[i];
        }
        if (delta >= ea || delta <= -eb) return false;
        if (axis == 3) return true;
        const int64_t s = stride[axis];
        if (s == 0) return meet(axis + 1, delta);
        // steps d from a's to b's, -na < d < nb, whose distance delta + d s is between what is left of b and of a
        const int64_t ra = ea - (na[axis] - 1) * s, rb = eb - (nb[axis] - 1) * s;
        const auto floor_div = [](int64_t x, int64_t y) { return x / y - (x % y < 0); };
        const int64_t low = std::max(1 - na[axis], floor_div(-rb - delta, s) + 1);
        const int64_t high = std::min(nb[axis] - 1, -floor_div(delta - ra, s) - 1);
        if (high - low > 3) return true;
        for (int64_t d = low; d <= high; ++d)
            if (meet(axis + 1, delta + d * s)) return true;
        return false;
    }
};

// Whether two fields share no memory: their extents do not meet, or both repeat with the same strides, of which the
// batch's is a multiple of the token's or the reverse, and no row of one is a row of the other.
// (Heads that are not as far apart in both count as one piece, gaps and all.)
bool apart(Field a, Field b) {
    if (!a.p || !b.p) return true;
    const Span x = span_of(a), y = span_of(b);
    if (!overlaps(x.p, x.bytes, y.p, y.bytes)) return true;
    if (a.n[1] > 1 && b.n[1] > 1 && a.stride[1] != b.stride[1])
        for (Field *f : {&a, &b}) {
            f->inner += (f->n[1] - 1) * f->stride[1];
            f->n[1] = 1;
        }
    Pair pair;
    int64_t stride[3];
    for (int i = 0; i < 3; ++i) {  // (an axis of one has no stride)
        if (a.n[i] > 1 && b.n[i] > 1 && a.stride[i] != b.stride[i]) return false;
        stride[i] = a.n[i] > 1 ? a.stride[i] : b.n[i] > 1 ? b.stride[i] : 0;
    }
    const int64_t low = std::min(stride[0], stride[2]), high = std::max(stride[0], stride[2]);
    if (low > 0 && high % low != 0) return false;
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int i, int j) { return stride[i] > stride[j]; });
    for (int i = 0; i < 3; ++i) {
        pair.na[i] = a.n[order[i]];
        pair.nb[i] = b.n[order[i]];
        pair.stride[i] = stride[order[i]];
    }
    pair.inner_a = a.inner;
    pair.inner_b = b.inner;
    const auto bytes = reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p);
    return !pair.meet(0, bytes / 2);
}

struct Rows {
    const void *p;
    int64_t heads, stride[3];  // batch, head, token

    Field field(int64_t B, int64_t S, int64_t D) const {
        Field f;
        f.p = p;
        const int64_t n[3] = {B, heads, S};
        std::copy(n, n + 3, f.n);
        std::copy(stride, stride + 3, f.stride);
        f.inner = D;
        return f;
    }
    bool same(const Rows &o) const {
        return p == o.p && heads == o.heads && std::equal(stride, stride + 3, o.stride);
    }
};

// A tensor of rows: its strides (the contiguous ones where none are given), looked over.  An output's rows
// may not share memory.
tsa_status rows_in(const void *p, const int64_t *strides, int64_t B, int64_t heads, int64_t S, int64_t D, bool output,
                   Rows *r) {
    *r = {p, heads, {0, 0, 0}};
    if (!p) return TSA_OK;
    const int64_t dense[3] = {heads * S * D, S * D, D}, n[3] = {B, heads, S};
    for (int i = 0; i < 3; ++i) {
        r->stride[i] = n[i] == 1 ? 0 : strides ? strides[i] : dense[i];
        if (r->stride[i] < 0 || r->stride[i] % 8 || r->stride[i] > kMaxExtent) return TSA_ERR_INVALID_ARGUMENT;
    }
    TSA_TRY(check_aligned({p}, 15));
    __int128 e = D;
    for (int i = 0; i < 3; ++i) e += (__int128)(n[i] - 1) * r->stride[i];
    if (e > kMaxExtent) return TSA_ERR_INVALID_ARGUMENT;
    if (!output) return TSA_OK;
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int x, int y) { return r->stride[x] < r->stride[y]; });
    int64_t taken = D;
    for (int i : order) {
        if (n[i] == 1) continue;
        if (r->stride[i] < taken) return TSA_ERR_INVALID_ARGUMENT;
        taken += (n[i] - 1) * r->stride[i];
    }
    return TSA_OK;
}

RowsPart part_of(const Rows &from, const Rows &to, bool rotated) {
    RowsPart p = {};
    p.from = static_cast<const uint16_t *>(from.p);
    p.to = static_cast<uint16_t *>(const_cast<void *>(to.p));
    p.from_batch = from.stride[0];
    p.from_head = from.stride[1];
    p.from_token = from.stride[2];
    p.to_batch = to.stride[0];
    p.to_head = to.stride[1];
    p.to_token = to.stride[2];
    p.heads = (int)from.heads;
    p.rotated = rotated;
    return p;
}

// A pair's turns per position, f / 2 pi, as a 64-bit fraction of a turn (modulo whole turns): the product with
// 1 / 2 pi in two binary64 parts, whose sum is off by less than 2^-100 turns times max(|f|, 1).
uint64_t fraction_of_turn(double f) {
    constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;  // 1 / 2 pi
    if (f < 0.0) return 0 - fraction_of_turn(-f);
    double p = f * kHi;
    const double e = std::fma(f, kHi, -p) + f * kLo;
    p -= std::floor(p);  // exact: p is not negative
    const double x = p * 0x1p64, whole = std::floor(x);
    return (uint64_t)whole + (uint64_t)(int64_t)std::llrint((x - whole) + e * 0x1p64);
}

tsa_status angles(const double *frequencies, int64_t R, int64_t D, float magnitude, bool back, RowsLaunch *a) {
    if (!std::isfinite(magnitude) || R <= 0) return TSA_ERR_INVALID_ARGUMENT;
    if (R % 16 || R > D) return TSA_ERR_UNSUPPORTED;
    // the frequencies are read here, on the host
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, frequencies) != cudaSuccess) (void)cudaGetLastError();
    else if (at.type == cudaMemoryTypeDevice) return TSA_ERR_INVALID_ARGUMENT;
    for (int64_t i = 0; i < R / 2; ++i) {
        if (!std::isfinite(frequencies[i]) || std::fabs(frequencies[i]) > 65536.0) return TSA_ERR_INVALID_ARGUMENT;
        const uint64_t f = fraction_of_turn(frequencies[i]);
        a->step[i] = back ? 0 - f : f;
    }
    a->R = (int)R;
    a->magnitude = magnitude;
    return TSA_OK;
}

tsa_status check_rows_shape(tsa_dtype dtype, int64_t B, int64_t S, int64_t D) {
    if (dtype != TSA_F16 && dtype != TSA_BF16) return TSA_ERR_INVALID_ARGUMENT;
    if (B <= 0 || S <= 0 || D <= 0) return TSA_ERR_INVALID_ARGUMENT;
    if (D % 16 || D > kMaxRotaryDim) return TSA_ERR_UNSUPPORTED;
    if (B > INT_MAX || S > INT_MAX || B * S > INT_MAX) return TSA_ERR_UNSUPPORTED;
    return TSA_OK;
}

tsa_status check_heads(int64_t heads) {
    return heads <= 0 ? TSA_ERR_INVALID_ARGUMENT : heads > 65535 ? TSA_ERR_UNSUPPORTED : TSA_OK;
}

// A paged cache's sizes; its arrays as fields.
struct Pages {
    Field k, v;
    int shift;
};

tsa_status pages_in(const void *K_cache, const void *V_cache, int64_t num_pages, int64_t page_size, int64_t k_stride,
                    int64_t v_stride, int64_t max_pages, int64_t HK, int64_t D, Pages *c) {
    if (num_pages <= 0 || page_size <= 0 || max_pages <= 0) return TSA_ERR_INVALID_ARGUMENT;
    if ((page_size & (page_size - 1)) || page_size < 16 || page_size > 256) return TSA_ERR_UNSUPPORTED;
    if (num_pages > INT_MAX || max_pages > (INT_MAX - 256) / page_size) return TSA_ERR_UNSUPPORTED;
    c->shift = 0;
    while ((1 << c->shift) < page_size) ++c->shift;
    TSA_TRY(check_aligned({K_cache, V_cache}, 15));
    const void *const p[2] = {K_cache, V_cache};
    const int64_t stride[2] = {k_stride, v_stride};
    Field *const f[2] = {&c->k, &c->v};
    for (int i = 0; i < 2; ++i) {
        f[i]->p = p[i];
        f[i]->n[0] = num_pages;
        f[i]->inner = HK * page_size * D;
        f[i]->stride[0] = num_pages == 1 ? f[i]->inner : stride[i];
        int64_t e;
        if (f[i]->stride[0] % 8 || f[i]->stride[0] < f[i]->inner || f[i]->stride[0] > kMaxExtent || !extent(*f[i], &e))
            return TSA_ERR_INVALID_ARGUMENT;
    }
    return TSA_OK;
}

tsa_status start(RowsLaunch *a, tsa_dtype dtype, int64_t B, int64_t S, int64_t D, int interleaved, int dev,
                 tsa_stream_t stream, int *sms) {
    a->B = (int)B;
    a->S = (int)S;
    a->D = (int)D;
    a->bf16 = dtype == TSA_BF16;
    a->interleaved = interleaved != 0;
    a->stream = reinterpret_cast<cudaStream_t>(stream);
    TSA_TRY(multiprocessors(dev, sms));
    return device_flags(dev, &a->flags);
}

tsa_status paged_decode_launch(int64_t B, int64_t H, int64_t HK, int64_t D, int64_t page_size, int64_t max_pages,
                               int64_t block, int64_t nnz_cap, PagedDecodeLaunch *a) {
    if (B <= 0 || H <= 0 || HK <= 0 || D <= 0 || block <= 0 || nnz_cap < 0 || page_size <= 0 || max_pages <= 0)
        return TSA_ERR_INVALID_ARGUMENT;
    if (H % HK) return TSA_ERR_INVALID_ARGUMENT;
    if ((block != 32 && block != 64 && block != 128) || (D != 64 && D != 128)) return TSA_ERR_UNSUPPORTED;
    if (B > 65535 || H > 65535 || B * H > 65535 || nnz_cap > INT_MAX / 4) return TSA_ERR_UNSUPPORTED;
    if ((page_size & (page_size - 1)) || page_size < 16 || page_size > 256 || max_pages > (INT_MAX - 256) / page_size)
        return TSA_ERR_UNSUPPORTED;
    a->B = (int)B;
    a->H = (int)H;
    a->HK = (int)HK;
    a->D = (int)D;
    a->block = (int)block;
    a->nnz_cap = (int)nnz_cap;
    a->max_pages = (int)max_pages;
    a->page_shift = 0;
    while ((1 << a->page_shift) < page_size) ++a->page_shift;
    split_paged_decode(a);
    return TSA_OK;
}

}  // namespace
}  // namespace tsa

using namespace tsa;

extern "C" {

tsa_status tsa_rotary(const void *Q, const void *K, const int64_t *strides, const int32_t *positions,
                      int64_t position_rows, const double *frequencies, int64_t rotary_dim, int interleaved,
                      float magnitude, int inverse, void *Q_out, void *K_out, tsa_dtype dtype, int64_t B, int64_t H,
                      int64_t HK, int64_t S, int64_t D, tsa_stream_t stream) {
    if (!Q || !Q_out || !frequencies || !K != !K_out) return TSA_ERR_INVALID_ARGUMENT;
    if (positions && position_rows != 1 && position_rows != B) return TSA_ERR_INVALID_ARGUMENT;
    TSA_TRY(check_rows_shape(dtype, B, S, D));
    TSA_TRY(check_heads(H));
    if (K) TSA_TRY(check_heads(HK));
    else HK = 1;
    RowsLaunch a = {};
    TSA_TRY(angles(frequencies, rotary_dim, D, magnitude, inverse != 0, &a));
    TSA_TRY(check_aligned({positions}, 3));
    Rows q, k, qo, ko;
    TSA_TRY(rows_in(Q, strides, B, H, S, D, false, &q));
    TSA_TRY(rows_in(K, strides ? strides + 3 : nullptr, B, HK, S, D, false, &k));
    TSA_TRY(rows_in(Q_out, strides ? strides + 6 : nullptr, B, H, S, D, true, &qo));
    TSA_TRY(rows_in(K_out, strides ? strides + 9 : nullptr, B, HK, S, D, K != nullptr, &ko));
    const Field fq = q.field(B, S, D), fk = k.field(B, S, D), fqo = qo.field(B, S, D), fko = ko.field(B, S, D);
    const Span at = {positions, (size_t)(position_rows * S) * 4}, oq = span_of(fqo), ok = span_of(fko);
    if ((!qo.same(q) && !apart(fqo, fq)) || !apart(fqo, fk) || !apart(fqo, fko) || (K && !ko.same(k) && !apart(fko, fk)) ||
        !apart(fko, fq) || outputs_overlap({oq}, {at}) || outputs_overlap({ok}, {at}))
        return TSA_ERR_INVALID_ARGUMENT;
    int dev, sms;
    TSA_TRY(current_device(&dev));
    TSA_TRY(check_device({Q, K, positions, Q_out, K_out}, dev));
    a.part[0] = part_of(q, qo, true);
    if (K) a.part[1] = part_of(k, ko, true);
    a.positions = positions;
    a.position_rows = (int)position_rows;
    TSA_TRY(start(&a, dtype, B, S, D, interleaved, dev, stream, &sms));
    return launch_rows(&a, sms);
}

tsa_status tsa_paged_append(const void *Q, const void *K, const void *V, const int64_t *strides, void *K_cache,
                            void *V_cache, int64_t num_pages, int64_t page_size, int64_t k_page_stride,
                            int64_t v_page_stride, const int32_t *page_table, int64_t max_pages,
                            const int32_t *seq_lens, const int32_t *counts, const double *frequencies,
                            int64_t rotary_dim, int interleaved, float magnitude, void *Q_out, tsa_dtype dtype,
                            int64_t B, int64_t H, int64_t HK, int64_t T, int64_t D, tsa_stream_t stream) {
    if (!K || !V || !K_cache || !V_cache || !page_table || !seq_lens || !Q != !Q_out || (Q && !frequencies))
        return TSA_ERR_INVALID_ARGUMENT;
    TSA_TRY(check_rows_shape(dtype, B, T, D));
    TSA_TRY(check_heads(HK));
    if (Q) TSA_TRY(check_heads(H));
    else H = 1;
    RowsLaunch a = {};
    if (frequencies) TSA_TRY(angles(frequencies, rotary_dim, D, magnitude, false, &a));
    Pages c;
    TSA_TRY(pages_in(K_cache, V_cache, num_pages, page_size, k_page_stride, v_page_stride, max_pages, HK, D, &c));
    TSA_TRY(check_aligned({page_table, seq_lens, counts}, 3));
    Rows q, k, v, qo;
    TSA_TRY(rows_in(Q, strides, B, H, T, D, false, &q));
    TSA_TRY(rows_in(K, strides ? strides + 3 : nullptr, B, HK, T, D, false, &k));
    TSA_TRY(rows_in(V, strides ? strides + 6 : nullptr, B, HK, T, D, false, &v));
    TSA_TRY(rows_in(Q_out, strides ? strides + 9 : nullptr, B, H, T, D, Q != nullptr, &qo));
    const Field fq = q.field(B, T, D), fk = k.field(B, T, D), fv = v.field(B, T, D), fqo = qo.field(B, T, D);
    const Span lists[3] = {{page_table, (size_t)(B * max_pages) * 4}, {seq_lens, (size_t)B * 4}, {counts, (size_t)B * 4}};
    if (!apart(c.k, c.v) || (Q && !qo.same(q) && !apart(fqo, fq))) return TSA_ERR_INVALID_ARGUMENT;
    const Field *const outs[3] = {&c.k, &c.v, &fqo};
    for (const Field *o : outs) {
        if (!apart(*o, fk) || !apart(*o, fv)) return TSA_ERR_INVALID_ARGUMENT;
        if (o != &fqo && (!apart(*o, fq) || !apart(*o, fqo))) return TSA_ERR_INVALID_ARGUMENT;
        if (outputs_overlap({span_of(*o)}, {lists[0], lists[1], lists[2]})) return TSA_ERR_INVALID_ARGUMENT;
    }
    int dev, sms;
    TSA_TRY(current_device(&dev));
    TSA_TRY(check_device({Q, K, V, K_cache, V_cache, page_table, seq_lens, counts, Q_out}, dev));
    const int64_t head = page_size * D;
    const Rows kc = {K_cache, HK, {0, head, 0}}, vc = {V_cache, HK, {0, head, 0}};
    if (Q) a.part[0] = part_of(q, qo, true);
    a.part[1] = part_of(k, kc, frequencies != nullptr);
    a.part[1].page_stride = c.k.stride[0];
    a.part[2] = part_of(v, vc, false);
    a.part[2].page_stride = c.v.stride[0];
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.counts = counts;
    a.num_pages = num_pages;
    a.max_pages = (int)max_pages;
    a.page_shift = c.shift;
    TSA_TRY(start(&a, dtype, B, T, D, interleaved, dev, stream, &sms));
    return launch_rows(&a, sms);
}

size_t tsa_paged_attention_decode_workspace_bytes(int64_t B, int64_t H, int64_t HK, int64_t D, int64_t page_size,
                                                  int64_t max_pages, int64_t block, int64_t nnz_cap) {
    PagedDecodeLaunch a = {};
    return paged_decode_launch(B, H, HK, D, page_size, max_pages, block, nnz_cap, &a) == TSA_OK ? paged_decode_workspace(a)
                                                                                             : 0;
}

tsa_status tsa_paged_attention_decode(const void *Q, const void *K_cache, const void *V_cache, int64_t num_pages,
                                      int64_t page_size, int64_t k_page_stride, int64_t v_page_stride,
                                      const int32_t *page_table, int64_t max_pages, const int32_t *seq_lens,
                                      const int32_t *row_ptr, const int32_t *col_idx, int64_t nnz_cap, void *O,
                                      tsa_dtype dtype, int64_t B, int64_t H, int64_t HK, int64_t D, int64_t block,
                                      float scale, void *workspace, size_t workspace_bytes, tsa_stream_t stream) {
    if (!Q || !K_cache || !V_cache || !page_table || !seq_lens || !O || !row_ptr != !col_idx || (!row_ptr && nnz_cap != 0) ||
        (row_ptr && nnz_cap < 1))
        return TSA_ERR_INVALID_ARGUMENT;
    if (dtype != TSA_F16 && dtype != TSA_BF16) return TSA_ERR_INVALID_ARGUMENT;
    if (!std::isfinite(scale) || scale < 1e-30f) return TSA_ERR_INVALID_ARGUMENT;
    PagedDecodeLaunch a = {};
    TSA_TRY(paged_decode_launch(B, H, HK, D, page_size, max_pages, block, nnz_cap, &a));
    Pages c;
    TSA_TRY(pages_in(K_cache, V_cache, num_pages, page_size, k_page_stride, v_page_stride, max_pages, HK, D, &c));
    TSA_TRY(check_aligned({Q, O}, 15));
    TSA_TRY(check_aligned({page_table, seq_lens, row_ptr, col_idx}, 3));
    TSA_TRY(check_aligned({workspace}, 255));
    const size_t need = paged_decode_workspace(a), one = (size_t)(B * H * D) * 2;
    if (need > 0 && !workspace) return TSA_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < need) return TSA_ERR_CAPACITY;
    if (outputs_overlap({{O, one}, {need > 0 ? workspace : nullptr, need}},
                        {{Q, one}, span_of(c.k), span_of(c.v), {page_table, (size_t)(B * max_pages) * 4},
                         {seq_lens, (size_t)B * 4}, rows_of(row_ptr, B, 1), entries_of(col_idx, nnz_cap)}))
        return TSA_ERR_INVALID_ARGUMENT;
    int dev;
    TSA_TRY(current_device(&dev));
    TSA_TRY(check_device({Q, K_cache, V_cache, page_table, seq_lens, row_ptr, col_idx, O}, dev));
    if (need > 0) TSA_TRY(check_device_ptr(workspace, dev));
    a.Q = static_cast<const uint16_t *>(Q);
    a.K = static_cast<const uint16_t *>(K_cache);
    a.V = static_cast<const uint16_t *>(V_cache);
    a.page_table = page_table;
    a.lens = seq_lens;
    a.row_ptr = row_ptr;
    a.col_idx = col_idx;
    a.k_page_stride = c.k.stride[0];
    a.v_page_stride = c.v.stride[0];
    a.O = static_cast<uint16_t *>(O);
    a.partial = static_cast<float *>(workspace);
    a.num_pages = (int)num_pages;
    a.bf16 = dtype == TSA_BF16;
    a.scale_log2 = (float)((double)scale * 1.4426950408889634);
    a.stream = reinterpret_cast<cudaStream_t>(stream);
    TSA_TRY(device_flags(dev, &a.flags));
    return launch_paged_decode(a);
}

}  // extern "C"
