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

// The buckets as a kernel keeps them in shared memory: biases in log2 units and starts, and, for kernels
// that call spread, the bias of each of the first distances.
constexpr int kDistances = 2048;  // 8 KB beside the D = 128 forward's tiles, two thread blocks per SM
constexpr int kDistFront = 64;    // distances below zero lie behind the causal mask; they may be read
struct BucketTable {
    float *bias;  // kMaxBuckets
    int *start;   // kMaxBuckets (INT_MAX from n on)
    float *dist;  // [-kDistFront, kDistances)

    __device__ __forceinline__ explicit BucketTable(uint8_t *smem)
        : bias(reinterpret_cast<float *>(smem)), start(reinterpret_cast<int *>(smem) + kMaxBuckets),
          dist(reinterpret_cast<float *>(smem) + 2 * kMaxBuckets + kDistFront) {}

    template <bool kBF16>
    __device__ __forceinline__ void load(const BiasTerms &t, int head, int tid, int nthreads) const {
        for (int b = tid; b < kMaxBuckets; b += nthreads) {
            bias[b] = b < t.n ? bias_log2(widen16<kBF16>(__ldg(t.bias + (long long)head * t.n + b))) : 0.f;
            start[b] = t.starts[b];
        }
    }

    // The last of n buckets that starts at or before distance d.
    __device__ __forceinline__ int find(int n, int d) const {
        int at = 0;
        for (int s = n > 1 ? 1 << (31 - __clz(n - 1)) : 0; s > 0; s >>= 1)
            if (start[min(at + s, kMaxBuckets - 1)] <= d) at += s;
        return at;
    }

    // After load and a barrier: fills dist up to where a step can still touch two buckets (or to
    // `limit`), four distances per thread at a time, each by halving.  Returns how many are known;
    // another barrier before they are read.
    __device__ __forceinline__ int spread(int n, int limit, int tid, int nthreads) const {
        for (int d = tid; d < kDistFront; d += nthreads) dist[d - kDistFront] = 0.f;
        int known = min(kDistances, limit);
        if (start[n - 1] < kDistances - 95) known = min(known, start[n - 1] + 95);
        const int first = n > 1 ? 1 << (31 - __clz(n - 1)) : 0;
        for (int d = tid; d < known; d += 4 * nthreads) {
            int at[4] = {0, 0, 0, 0};
            for (int s = first; s > 0; s >>= 1)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    if (start[min(at[x] + s, kMaxBuckets - 1)] <= d + x * nthreads) at[x] += s;
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (d + x * nthreads < known) dist[d + x * nthreads] = bias[at[x]];
        }
        return known;
    }
};
constexpr int kBucketBytes = 2 * kMaxBuckets * 4;  // without the distances
constexpr int kBucketTableBytes = kBucketBytes + (kDistFront + kDistances) * 4;

// One warp's 32 rows x 64 columns of a step hold 95 distances, d_lo .. d_lo + 94 (negative ones
// lie behind the causal mask).
constexpr int kWindow = 96;

// The biases of the distances d_lo + 0 .. 94, which may lie in several buckets: the table's, or, beyond
// it, laid out in `win` (three entries per lane, and a walk down the n buckets that is the same in all
// lanes).
__device__ __forceinline__ const float *window_at(float *win, const BucketTable &t, int known, int n, int d_lo,
                                                  int lane) {
    if (d_lo + kWindow - 2 < known) return t.dist + d_lo;
    const int top = t.find(n, d_lo + kWindow - 2);
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
    return win;
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
