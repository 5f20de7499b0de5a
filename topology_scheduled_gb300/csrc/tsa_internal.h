// tsa_internal.h -- declarations shared by the library's translation units (not installed).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "score_terms.cuh"
#include "tsa.h"
#include "tsa_device.cuh"

namespace tsa {

// Host side of every call (api.cu).
#define TSA_TRY(expr)                       \
    do {                                    \
        const tsa_status s_ = (expr);       \
        if (s_ != TSA_OK) return s_;        \
    } while (0)
tsa_status current_device(int *dev);
tsa_status device_flags(int dev, DeviceFlags *f);
tsa_status check_device_ptr(const void *p, int dev);
tsa_status multiprocessors(int dev, int *sms);
// Row-major 16-bit tensor [lanes, rows, cols]; boxes of 64 columns x box_rows, cut off at a lane's end.
bool encode_3d(CUtensorMap *map, const void *ptr, bool bf16, uint64_t lanes, uint64_t rows, uint64_t cols,
               uint32_t box_rows);
bool overlaps(const void *a, size_t na, const void *b, size_t nb);

// Lets `kernel` have `bytes` of dynamic shared memory on the current device.  `done` (one per kernel and
// size) keeps a bit per device, so only the first call asks the driver, which takes about a microsecond.
inline bool allow_smem(std::atomic<unsigned long long> &done, const void *kernel, int bytes) {
    int dev;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (done.load(std::memory_order_relaxed) & bit) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

struct AttnLaunch {
    const CUtensorMap *tmQ, *tmK, *tmV, *tmO;
    const CUtensorMap *tmO2;  // differential: the second map's output (otherwise tmO again)
    const int32_t *row_ptr, *col_idx;
    int nnz_cap;  // entries of col_idx (read with score terms only)
    bool with_o2;  // differential: the second map's output is wanted
    float *lse;  // optional: natural-log log-sum-exp of the scaled scores per query row
    int nb, S, D, lanes;  // nb: 64-token blocks
    bool bf16;
    int gran;  // token block of the CSR: 0 for 64, 1 for 128, 2 for 32
    float scale_log2;
    DeviceFlags flags;
    cudaStream_t stream;
};

tsa_status launch_scheduled_attention(const AttnLaunch &a);
tsa_status launch_biased_attention(const AttnLaunch &a, const BiasTerms &terms);
tsa_status launch_differential_attention(const AttnLaunch &a, const DiffTerms &terms);

// Byte offsets of the backward pass's workspace regions (each 256-byte aligned).
struct BwdWorkspace {
    size_t delta, lse_pad, vlen, cnt, col_ptr, bitmap, bitmap_bytes, row_idx, pairs, vlen_in, rp64, ci64, total;
};
// nb: 64-token blocks; nb_in: rows of a 128-token CSR to expand first (0: the CSR is 64-token)
BwdWorkspace backward_workspace_layout(int64_t lanes, int64_t S, int64_t nb, int64_t nnz_cap, int64_t nb_in);

// Largest number of query blocks the backward pass accepts (its column bitmap is nb^2 bits).
constexpr int64_t kMaxBackwardBlocks = 8192;

struct BwdLaunch {
    // 128-row boxes (tiles resident in a CTA) and 64-row boxes (streamed blocks, stores)
    const CUtensorMap *tmQ128, *tmdO128;
    const CUtensorMap *tmQ64, *tmdO64, *tmK64, *tmV64, *tmdQ64, *tmdK64, *tmdV64;
    const uint16_t *O, *dO;
    const float *lse;
    const int32_t *row_ptr, *col_idx;
    int64_t nnz_cap;
    long long read_cap;  // entries of col_idx that may be read
    float *partial;      // score terms: each tile's part of the learned inputs' gradients
    // Delta and the log-sum-exp per lane over nb * 64 rows, so a partial last block is read like any
    // other; the log-sum-exp in log2 units, +inf for rows past S and rows without keys
    float *delta, *lse_pad;
    int *vlen, *cnt, *col_ptr;
    unsigned *bitmap;
    size_t bitmap_bytes;
    int32_t *row_idx;
    int *pairs;  // dK/dV key-block pairs, 2 per pair (-1: none)
    int nb_in;   // > 0: row_ptr/col_idx are a CSR of nb_in 128-token blocks, expanded into
    int *vlen_in;  // rp64/ci64 (64-token blocks, capacity nnz_cap) before anything else
    int32_t *rp64, *ci64;
    int nb, S, D, lanes;
    bool bf16;
    float scale;
    DeviceFlags flags;
    cudaStream_t stream;
};

tsa_status launch_attention_backward(const BwdLaunch &a);
// Its first launches: the transposed schedule (a 128-token CSR is replaced by its expansion in *a),
// and Delta with the log-sum-exp in padded rows.  A short schedule's transpose is built by the second.
struct SmallSchedule;
SmallSchedule small_schedule(const BwdLaunch &a);  // nb 0: the schedule is not short
tsa_status launch_backward_schedule(BwdLaunch *a);
tsa_status launch_backward_delta(const BwdLaunch &a);

// Backward passes with score terms.  dbias [H, n]; dlambda: the gradients of lq1, lk1, lq2, lk2.
tsa_status launch_biased_backward(const BwdLaunch &a, const BiasTerms &terms, uint16_t *dbias);
tsa_status launch_differential_backward(const BwdLaunch &a, const DiffTerms &terms, const uint16_t *O2,
                                        uint16_t *const dlambda[4]);

// One new token per sequence against a cache [lanes, cap, D], lanes = B * H; row_ptr has B + 1 entries.
struct DecodeLaunch {
    const uint16_t *Q, *K, *V;
    const int32_t *lens, *row_ptr, *col_idx;
    int nnz_cap;
    uint16_t *O;
    int lanes, H, cap, D, block, sms;
    bool bf16;
    float scale_log2;
    DeviceFlags flags;
    cudaStream_t stream;
};

tsa_status launch_biased_decode(const DecodeLaunch &a, const BiasTerms &terms);
tsa_status launch_differential_decode(const DecodeLaunch &a, const DiffTerms &terms);

// Largest number of blocks the schedule builder accepts.
constexpr int64_t kMaxScheduleBlocks = 4096;
constexpr int64_t kMaxScheduleDim = 1024;

// Byte offsets of the builder's workspace regions (each 256-byte aligned).
struct ScheduleWorkspace {
    size_t part, cent, cent32, bnd, comp, vb_d, vb_u, mst_d, mst_u, mst_v, counters, sal, cnt, perm, sal_rank, gbar, total;
};
ScheduleWorkspace schedule_workspace_layout(int64_t lanes, int64_t nb, int64_t D);

struct ScheduleLaunch {
    const uint16_t *K;
    bool bf16;
    int64_t lanes, S, D, block, nb;
    int64_t sink, local_radius, topk;
    bool content_ties;  // break ties by centroid content instead of block index
    int32_t *row_ptr, *col_idx;
    int64_t col_cap;
    double *salience_sq;  // may be null
    uint8_t *workspace;
    DeviceFlags flags;
    cudaStream_t stream;
};

tsa_status launch_build_schedule(const ScheduleLaunch &a);
// The two halves of launch_build_schedule, for a lane-sharded build: per-lane block sums of K
// (part: lanes x nb x D doubles), and the schedule from block sums of all lanes.
tsa_status launch_block_sums(const ScheduleLaunch &a, double *part);
tsa_status launch_schedule_from_sums(const ScheduleLaunch &a, const double *sums);
tsa_status launch_dense_causal_csr(int64_t nb, int32_t *row_ptr, int32_t *col_idx,
                                   cudaStream_t stream);
// Segment schedule: fixed segments of seg_tokens (> 0), or the listed starts (seg_tokens 0).
tsa_status launch_segment_csr(int64_t S, int64_t block, int64_t seg_tokens, const int32_t *starts,
                              int64_t n_starts, int32_t *row_ptr, int32_t *col_idx, int64_t col_cap,
                              const DeviceFlags &flags, cudaStream_t stream);

}  // namespace tsa
