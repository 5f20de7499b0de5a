// score_terms.cuh -- what the attention kernels add to the plain scheduled softmax: nothing, a
// learned bias per head and bucket of the distance q - k, or a second softmax map that is
// subtracted with a learned weight.  The kernels take one of these types as a template argument
// and as their last parameter (by value, read from the constant bank).
#pragma once

#include <stdint.h>

#include "tsa_device.cuh"
#include "tsa_terms.h"

namespace tsa {

constexpr int kMaxBuckets = TSA_MAX_BUCKETS;

// softmax(scale q.k): the scheduled attention itself.
struct NoTerms {
    static constexpr bool kBias = false, kDiff = false;
};

// softmax(scale q.k + bias[head, bucket(q - k)]): bucket b holds the distances from starts[b] up
// to the next start; the last one is open.
struct BiasTerms {
    static constexpr bool kBias = true, kDiff = false;
    const uint16_t *bias;  // [H, n], the inputs' type
    int H, n;
    int32_t starts[kMaxBuckets];  // ascending, starts[0] == 0
};

// softmax(scale q1.k1) - lambda softmax(scale q2.k2), q1 | q2 and k1 | k2 the halves of a row,
// lambda = exp(lq1.lk1) - exp(lq2.lk2) + init.
struct DiffTerms {
    static constexpr bool kBias = false, kDiff = true;
    const uint16_t *lq1, *lk1, *lq2, *lk2;  // [H or 1, D / 2], the inputs' type
    int H, per_head;                        // per_head 0: one lambda for every head
    float init;
    long long map_rows;  // rows of one map in the per-row arrays (log-sum-exp, Delta)
};

// A bias this low leaves its keys out, as -inf does: adding the lowest value of bf16 to a score is
// a mask, and its product with log2(e) would be -inf in binary32 anyway.
constexpr float kBiasOut = -1e30f;

__device__ __forceinline__ float bias_log2(float b) {
    return b <= kBiasOut ? -INFINITY : b * 1.4426950408889634f;
}

// The buckets as a kernel keeps them in shared memory: biases in log2 units and starts.
struct BucketTable {
    float *bias;  // kMaxBuckets
    int *start;   // kMaxBuckets

    template <bool kBF16>
    __device__ __forceinline__ void load(const BiasTerms &t, int head, int tid, int nthreads) const {
        for (int b = tid; b < t.n; b += nthreads) {
            bias[b] = bias_log2(widen16<kBF16>(__ldg(t.bias + (long long)head * t.n + b)));
            start[b] = t.starts[b];
        }
    }
};
constexpr int kBucketTableBytes = kMaxBuckets * 8;

// One warp's 32 rows x 64 columns of a step hold 95 distances, d_lo .. d_lo + 94 (negative ones
// lie behind the causal mask).
constexpr int kWindow = 96;

// Fills win[0 .. 95] with the biases of the distances d_lo + 0 .. 95; `top` is the bucket of the
// largest one.  Three entries per lane, and a walk down the buckets that is the same in all lanes.
__device__ __forceinline__ void fill_window(float *win, const BucketTable &t, int top, int d_lo, int lane) {
    const int d0 = d_lo + lane, d1 = d0 + 32, d2 = d0 + 64;
    const int least = d_lo > 0 ? d_lo : 0;
    float w0 = t.bias[top], w1 = w0, w2 = w0;
    for (int b = top; b > 0 && t.start[b] > least; --b) {
        const int s = t.start[b];
        const float v = t.bias[b - 1];
        w0 = d0 < s ? v : w0;
        w1 = d1 < s ? v : w1;
        w2 = d2 < s ? v : w2;
    }
    win[lane] = w0;
    win[lane + 32] = w1;
    win[lane + 64] = w2;
    __syncwarp();
}

// lambda of `head`, by the whole warp: each lane multiplies kW / 32 pairs of each product (kW = D / 2).
template <int kW, bool kBF16>
__device__ __forceinline__ float lambda_of(const DiffTerms &t, int head, float *e1_out = nullptr,
                                           float *e2_out = nullptr) {
    const long long at = (t.per_head ? (long long)head * kW : 0) + (threadIdx.x & 31) * (kW / 32);
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int x = 0; x < kW / 32; ++x) {
        a = fmaf(widen16<kBF16>(__ldg(t.lq1 + at + x)), widen16<kBF16>(__ldg(t.lk1 + at + x)), a);
        b = fmaf(widen16<kBF16>(__ldg(t.lq2 + at + x)), widen16<kBF16>(__ldg(t.lk2 + at + x)), b);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, off);
        b += __shfl_xor_sync(0xffffffffu, b, off);
    }
    const float e1 = expf(a), e2 = expf(b);
    if (e1_out) { *e1_out = e1; *e2_out = e2; }
    return e1 - e2 + t.init;
}

// Loads and stores of a box of rows: a term's kernels see [lanes, S, D] as three dimensions, so
// that rows past a lane's end read as zero and are never written; the plain kernels keep theirs.
template <class Terms>
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap *map, int x, int row0, int y, int lane,
                                          uint32_t bar) {
    if constexpr (Terms::kBias || Terms::kDiff) tma_load_3d(dst, map, x, y, lane, bar);
    else tma_load_2d(dst, map, x, row0 + y, bar);
}

// Makes a 128-row tile of two copies of the same 64 rows block-diagonal: rows 0-63 keep the first
// half of their columns, rows 64-127 the second, so that one product with [x1 | x2] gives x1 in
// the upper and x2 in the lower rows.  `row` is the calling thread's (0-127); SW128 layout.
template <int D>
__device__ __forceinline__ void keep_diagonal(uint32_t tile, int row) {
    const uint32_t sw = (uint32_t)(row & 7);
    const int other = row >> 6 ? 0 : 1;  // the half to clear
    if constexpr (D == 128) {
#pragma unroll
        for (uint32_t u = 0; u < 8; ++u) st_shared_v4(tile + other * 16384 + row * 128 + u * 16, 0, 0, 0, 0);
    } else {
#pragma unroll
        for (uint32_t u = 0; u < 4; ++u)
            st_shared_v4(tile + row * 128 + (((other * 4 + u) ^ sw) << 4), 0, 0, 0, 0);
    }
}

}  // namespace tsa
