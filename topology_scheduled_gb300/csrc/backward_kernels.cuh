// backward_kernels.cuh -- the two gradient kernels of the scheduled causal attention on tcgen05
// tensor cores (sm_103a), plain or with the score terms of score_terms.cuh.  backward.cu has the
// mathematics and the launches around them.
//
// Bias by buckets.  P is recomputed with the bias, a constant per step or a window per warp as in the
// forward.  Its gradient sums dS over buckets in bwd_dq_kernel, in binary32 before dS is rounded:
//  * where a step touches a bucket before the last a warp adds up the diagonals of its values, one
//    distance each: for column c every lane takes the value of the row c + 1 lanes on (by a shuffle),
//    which lies on a diagonal of its own for all columns.  The sums of the first 256 distances wait in
//    shared memory until the tile is done; farther ones are added up by bucket at once, by shuffles too;
//  * the last, open bucket gets minus the sum of the row's other values, since a row of dS sums to
//    zero: almost no work on the far steps, and none of the error that Delta's rounded output leaves in
//    each of their many values (it is a common shift of a row's dP, which the far keys would add up).
//    In a row where every dS of the bucket is 0 (its bias a finite mask) it gets nothing.
// No atomics: a warp has its own sums, a CTA writes its tile's, and terms_reduce_bias adds the tiles
// in order.  Measured at [1, 32, 32768, 128] bf16, 14.5 blocks a row: dQ 880 us, dK/dV 1044 us (850 and
// 954 TFLOP/s on the three and four block products each does; the plain kernels, 64 lanes: 1435 and
// 1864 us).  Leaving a bucket without weight alone took the whole pass from 2036 to 2047 us.
//
// Differential attention.  A CTA takes a pair of blocks as the plain kernels do, and both maps of them:
// the first half of the score product's K steps goes into one accumulator, the second half into
// another, so the two maps' scores cost what a plain score does, and dP serves both maps.  The
// elementwise warps form dS1 and dS2 (= -lambda P2 o (dP - Delta2)); dQ and dK get each map's half of
// their columns from products of half the width, and dV one product with P1 - lambda P2, combined in
// binary32 and rounded once.  (Against one block per CTA with both maps in its 128 rows, by block-
// diagonal operands: 32 lanes of S 32768, topology, backward 3.36 -> 2.45 ms.)  lambda's gradient is
// - sum P2 o dP, summed over a CTA's rows in binary32 from the exact weights, so that a sum over every
// query keeps the precision that P's rounding would cost.  Measured there: dQ 885 us, dK/dV 1339 us (its
// dV product takes P from shared memory, as three accumulators and a step's products fill TMEM).
//
// What bounds the kernels: the tensor pipe is active for 22 to 37 % of the time and issue slots for 35 to
// 46 %.  One CTA holds all 512 TMEM columns, so a tile's prologue and epilogue stand alone on an SM, and a
// step's chain of products, elementwise work and accumulation is longer than its longest part.  P and dS
// are rounded to the inputs' type for their products: tcgen05 multiplies 16-bit operands at twice the
// rate of the 32-bit ones, which keep 10 bits.
#pragma once

#include <climits>
#include <type_traits>

#include "score_terms.cuh"
#include "tsa_device.cuh"
#include "tsa_internal.h"

namespace tsa {

// Where a short schedule's transpose comes from and goes to (see build_small_schedule).
struct SmallSchedule {
    int nb;  // 0: built elsewhere
    const int32_t *row_ptr, *col_idx;
    long long read_cap, cap;
    int *vlen, *col_ptr, *pairs;
    int32_t *row_idx;
    DeviceFlags flags;
};

namespace {

constexpr int kBlock = 64;
constexpr int kRows = 128;
constexpr int kEltWarps = 8;                   // elementwise warps: one per 32 rows x 32 columns of a step
constexpr int kElt = 32 * kEltWarps;
constexpr int kThreads = kElt + 64;
constexpr int kProducerWarp = kEltWarps;
constexpr int kMmaWarp = kEltWarps + 1;
constexpr int kStream = 4;     // depth of the ring of streamed blocks (what shared memory leaves)
constexpr int kMetaRing = 8;   // > kStream: a slot is rewritten only after its step is consumed
constexpr float kLog2e = 1.4426950408889634f;

// ---------------------------------------------------------------- shared helpers

// Two floats rounded to the 16-bit input dtype and packed (first in the low half).
template <bool kBF16>
__device__ __forceinline__ uint32_t pack16x2(float a, float b) {
    if constexpr (kBF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// The log-sum-exp as the gradient kernels subtract it: log2 units, and +inf for a row without keys,
// whose weights 2^(z - inf) are then 0 like those of rows past the end.
__device__ __forceinline__ float padded_lse(float lse) { return lse == -INFINITY ? INFINITY : lse * kLog2e; }

// The transposed schedule of a short 64-token CSR (at most kSmallBlocks rows), by one thread block of
// 256: what bwd_rows, bwd_col_count, bwd_col_scan, bwd_col_fill and bwd_col_pairs (backward.cu) write,
// with the bitmap in shared memory.  It runs beside the blocks that compute Delta, so a short sequence
// pays one launch instead of seven ([2, 8, 1000, 64]: 22 us of small launches).  Longer schedules keep
// the launches of their own: one block would read their rows one after another.
constexpr int kSmallBlocks = 64;
__device__ __forceinline__ void build_small_schedule(const SmallSchedule &g) {
    __shared__ unsigned bits[kSmallBlocks][kSmallBlocks / 32];
    __shared__ int count[kSmallBlocks], first[kSmallBlocks + 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nb = g.nb;
    for (int x = tid; x < kSmallBlocks * (kSmallBlocks / 32); x += blockDim.x) (&bits[0][0])[x] = 0u;
    __syncthreads();
    for (int i = warp; i < nb; i += blockDim.x >> 5) {  // a row per warp, as in bwd_rows
        const int b = g.row_ptr[i], len = g.row_ptr[i + 1] - b;
        int valid = 0;
        if (len >= 0 && len <= i + 1 && b >= 0 && (long long)b + len <= g.read_cap) {
            valid = len;
            for (int e0 = 0; e0 < valid; e0 += 32) {
                const int e = e0 + lane;
                bool bad = false;
                int j = 0;
                if (e < len) {
                    j = g.col_idx[b + e];
                    const int prev = e > 0 ? g.col_idx[b + e - 1] : -1;
                    bad = j < 0 || j > i || j <= prev;
                }
                const unsigned m = __ballot_sync(0xffffffffu, bad);
                if (m) valid = e0 + __ffs(m) - 1;
                if (e < valid) atomicOr(&bits[j][i >> 5], 1u << (i & 31));
            }
        }
        if (lane == 0) {
            if (valid != len) raise_status(g.flags, kDevBadSchedule);
            g.vlen[i] = valid;
        }
    }
    __syncthreads();
    if (tid < kSmallBlocks) count[tid] = tid < nb ? __popc(bits[tid][0]) + __popc(bits[tid][1]) : 0;
    __syncthreads();
    if (warp == 0) {  // exclusive scan, two columns per lane
        const int a = count[2 * lane], both = a + count[2 * lane + 1];
        int incl = both;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += x;
        }
        const bool fits = __shfl_sync(0xffffffffu, incl, 31) <= g.cap;
        if (lane == 0 && !fits) raise_status(g.flags, kDevCapacity);
        first[2 * lane] = fits ? incl - both : 0;
        first[2 * lane + 1] = fits ? incl - both + a : 0;
        if (lane == 31) first[kSmallBlocks] = fits ? incl : 0;
    }
    __syncthreads();
    for (int j = tid; j < nb; j += blockDim.x) {
        int at = first[j];
        const int end = first[j + 1];
        g.col_ptr[j] = at;
        if (j == nb - 1) g.col_ptr[nb] = end;
        for (int w = 0; w < kSmallBlocks / 32; ++w)
            for (unsigned m = bits[j][w]; m && at < end; m &= m - 1u) g.row_idx[at++] = w * 32 + __ffs(m) - 1;
        // the column's place by length (longest first), then by index
        int place = 0;
        for (int x = 0; x < nb; ++x) place += count[x] > count[j] || (count[x] == count[j] && x < j);
        g.pairs[place] = j;
        if (j == 0 && (nb & 1)) g.pairs[nb] = -1;
    }
}

// Union of two ascending index lists (already checked), with membership bits (1: first list,
// 2: second list); -1 at the end.
struct ListUnion {
    const int32_t *a, *b;
    int ia, ia_end, ib, ib_end;

    __device__ int next(int &flags) {
        const int ja = ia < ia_end ? __ldg(a + ia) : INT_MAX;
        const int jb = ib < ib_end ? __ldg(b + ib) : INT_MAX;
        if (ja == INT_MAX && jb == INT_MAX) {
            flags = 0;
            return -1;
        }
        const int j = ja < jb ? ja : jb;
        flags = (ja == j ? 1 : 0) | (jb == j ? 2 : 0);
        if (ja == j) ++ia;
        if (jb == j) ++ib;
        return j;
    }
};

// The epilogue's columns go 32 at a time; the two warps of a quarter of the rows (group 0 and 1) take
// half of the column blocks each.
//
// 128 rows of fp32 accumulator in TMEM (this warp's 32 lanes, D columns starting at `col`),
// times `mul`, rounded and written to a 128-row SW128 staging tile in the layout TMA stores.
template <int D, bool kBF16>
__device__ __forceinline__ void stage_rows(uint32_t tmem_row, uint32_t col, bool valid, float mul,
                                           uint32_t tile, int row, int group) {
    const uint32_t sw = (uint32_t)(row & 7);
#pragma unroll
    for (int x = 0; x < D / 64; ++x) {
        const int h = group * (D / 64) + x;
        uint32_t o[32];
        if (valid) {
            tmem_ld32(tmem_row + col + h * 32, o);
        } else {
#pragma unroll
            for (int t = 0; t < 32; ++t) o[t] = 0u;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int t = 0; t < 4; ++t)
                w[t] = pack16x2<kBF16>(__uint_as_float(o[q * 8 + 2 * t]) * mul,
                                       __uint_as_float(o[q * 8 + 2 * t + 1]) * mul);
            st_shared_v4(tile + (h >> 1) * 16384 + row * 128 + (((uint32_t)((h & 1) * 4 + q) ^ sw) << 4), w[0], w[1],
                         w[2], w[3]);
        }
    }
}

// Meta area (byte offsets from the meta base), common to both kernels.
constexpr int kBarTile = 0;                           // resident tile(s) loaded
constexpr int kBarFull = 8;                           // kStream x 8: streamed block landed
constexpr int kBarEmpty = kBarFull + 8 * kStream;     // kStream x 8: streamed block released
constexpr int kBarSFull = kBarEmpty + 8 * kStream;    // 2 x 8: products of a step in TMEM
constexpr int kBarPFull = kBarSFull + 16;             // 2 x 8: elementwise results of a step in TMEM
constexpr int kBarDone = kBarPFull + 16;              // 2 x 8: accumulation MMA of a step completed
constexpr int kBarFin = kBarDone + 16;
constexpr int kBarVFull = kBarFin + 8;                // dQ kernel: kStream x 8, V of a step landed
constexpr int kBarVEmpty = kBarVFull + 8 * kStream;   // dQ kernel: kStream x 8
constexpr int kBarLoaded = kBarVEmpty + 8 * kStream;  // dK/dV kernel, differential: 2 x 8, a step's products read
constexpr int kTmemSlot = kBarLoaded + 16;
constexpr int kAbortFlag = kTmemSlot + 4;
constexpr int kMetaJ = kAbortFlag + 4;                // kMetaRing x 4
constexpr int kMetaF = kMetaJ + 4 * kMetaRing;        // kMetaRing x 4
constexpr int kMetaBytes = 512;
static_assert(kMetaF + 4 * kMetaRing <= kMetaBytes, "meta area");

constexpr uint32_t kTmemCols = 512;  // S0 | S1 | dP0 | dP1 | accumulator(s)

// Each CTA takes all 512 TMEM columns, so a second CTA on the same SM would only wait in its
// allocation: ask for more than half of the SM's shared memory so that one CTA fits.
constexpr int smem_bytes_one_cta(int need) { return need > 116 * 1024 ? need : 116 * 1024; }
__device__ __forceinline__ uint32_t s_col(int b) { return b ? 64u : 0u; }
__device__ __forceinline__ uint32_t dp_col(int b) { return b ? 192u : 128u; }
constexpr uint32_t kAccCol = 256;
// dQ kernel, differential: S1 0 | 1, S2 0 | 1, dP 0 | 1, accumulator
__device__ __forceinline__ uint32_t s2_col(int b) { return b ? 192u : 128u; }
__device__ __forceinline__ uint32_t diff_dp_col(int b) { return b ? 320u : 256u; }
constexpr uint32_t kDiffAccCol = 384;
// dK/dV kernel, differential: the columns of product x of step u
__device__ __forceinline__ uint32_t diff_slot(int u, int x) { return (uint32_t)((3 * u + x) & 3) * 64u; }
// Elements 16 kk .. 16 kk + 15 of a step's packed results: each warp writes its 32 over its own 32
// columns of the products.
__device__ __forceinline__ constexpr uint32_t packed_col(int kk) { return (uint32_t)((kk >> 1) * 32 + (kk & 1) * 8); }

// ---------------------------------------------------------------- dQ
// Adds a warp's sums of dS per distance to its bucket sums, but for the last bucket's.  A lane's
// distances are d_lo + lane (a0), + 32 (a1) and + 64 (a2); `top` is the bucket of d_hi, `win` scratch
// (96 floats).
__device__ __forceinline__ void add_distances(float *bins, float *win, float a0, float a1, float a2,
                                              const BucketTable &t, int top, int last, int d_lo, int d_hi, int lane) {
    // running sums over the 96 distances that begin anew with each bucket (so that a bucket's sum
    // holds nothing of another's): where buckets begin, as three words of bits
    const int least = d_lo > 0 ? d_lo : 0;
    uint32_t m0 = 0u, m1 = 0u, m2 = 0u;
    for (int b0 = top; b0 > 0; b0 -= 32) {  // 32 buckets at a time, one per lane
        const int b = b0 - lane, at = b > 0 ? t.start[b] - d_lo : 0;
        const bool in = b > 0 && t.start[b] > least;
        const uint32_t bit = in ? 1u << (at & 31) : 0u;
        m0 |= __reduce_or_sync(0xffffffffu, at < 32 ? bit : 0u);
        m1 |= __reduce_or_sync(0xffffffffu, at >= 32 && at < 64 ? bit : 0u);
        m2 |= __reduce_or_sync(0xffffffffu, at >= 64 ? bit : 0u);
        if (!__all_sync(0xffffffffu, in)) break;
    }
    const uint32_t upto = 0xffffffffu >> (31 - lane);
    const int p0 = 31 - __clz(m0 & upto), p1 = 31 - __clz(m1 & upto), p2 = 31 - __clz(m2 & upto);  // -1: none
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float x0 = __shfl_up_sync(0xffffffffu, a0, o), x1 = __shfl_up_sync(0xffffffffu, a1, o),
                    x2 = __shfl_up_sync(0xffffffffu, a2, o);
        if (lane >= o && lane - o >= p0) a0 += x0;
        if (lane >= o && lane - o >= p1) a1 += x1;
        if (lane >= o && lane - o >= p2) a2 += x2;
    }
    const float c1 = __shfl_sync(0xffffffffu, a0, 31);
    if (p1 < 0) a1 += c1;
    const float c2 = __shfl_sync(0xffffffffu, a1, 31);
    if (p2 < 0) a2 += c2;
    win[lane] = a0;
    win[lane + 32] = a1;
    win[lane + 64] = a2;
    __syncwarp();
    // buckets top, top - 1, .. down to the one that holds the least distance, one per lane
    for (int b = top - lane; b >= 0; b -= 32) {
        const int end = b == top ? d_hi + 1 : t.start[b + 1];  // one past the bucket's last distance here
        if (end <= least) break;
        if (b != last && end > t.start[b]) bins[b] += win[end - 1 - d_lo];
    }
}

// A warp keeps the sums of dS of the first distances one by one until its tile is done; farther ones go
// to its bucket sums step by step.
constexpr int kNearSums = 256;
// A warp's row of them: distances below zero lie behind the mask, and a step whose farthest distance is the
// last one kept has its last lane add a 0 one place on.
constexpr int kNearRow = kDistFront + kNearSums + 1;

template <int D, class Terms>
struct DqSmem {
    static constexpr int kChunks = D / 64;
    static constexpr int kTileBytes = kRows * D * 2;   // Q and dO tiles (128 rows)
    static constexpr int kKVBytes = kBlock * D * 2;    // one K or V block
    static constexpr int kOffQ = 0;
    static constexpr int kOffDO = kOffQ + kTileBytes;
    static constexpr int kOffK = kOffDO + kTileBytes;
    static constexpr int kOffV = kOffK + kStream * kKVBytes;
    static constexpr int kOffMeta = kOffV + kStream * kKVBytes;
    static constexpr int kOffTable = kOffMeta + kMetaBytes;                      // bias only, up to kOffEnd
    static constexpr int kOffWin = kOffTable + kBucketTableBytes;                // a window of each warp
    static constexpr int kOffBins = kOffWin + kEltWarps * kWindow * 4;           // kMaxBuckets sums of each warp
    static constexpr int kOffNear = kOffBins + kEltWarps * kMaxBuckets * 4;      // sums by distance of each warp
    static constexpr int kEnd = Terms::kBias ? kOffNear + kEltWarps * kNearRow * 4 : kOffTable;
    static constexpr int kBytes = smem_bytes_one_cta(kEnd + 1024);  // + alignment slack
};

// partial: with a bias the tile's sums of dS per bucket, [lanes, tiles, n]; differential: the tile's
// part of lambda's gradient, [lanes, tiles].
template <int D, bool kBF16, class Terms>
__global__ void __launch_bounds__(kThreads, 1)
bwd_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmdO,
              const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
              const __grid_constant__ CUtensorMap tmdQ, const int32_t *__restrict__ row_ptr,
              const int32_t *__restrict__ col_idx, const int *__restrict__ vlen,
              const float *__restrict__ lse, const float *__restrict__ delta, int nb, float scale,
              float scale_log2, float *__restrict__ partial,
              DeviceFlags flags, const __grid_constant__ Terms terms) {
    constexpr bool kBias = Terms::kBias, kDiff = Terms::kDiff;
    using L = DqSmem<D, Terms>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_base = smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    if (base - raw_base + L::kEnd > (uint32_t)L::kBytes) {
        if (threadIdx.x == 0) raise_status(flags, kDevSmemAlign);
        return;
    }
    uint8_t *smem = smem_raw + (base - raw_base);
    [[maybe_unused]] const BucketTable table(smem + L::kOffTable);
    const uint32_t sQ = base + L::kOffQ, sdO = base + L::kOffDO, sK = base + L::kOffK, sV = base + L::kOffV;
    const uint32_t meta = base + L::kOffMeta;
    volatile int *meta_j = reinterpret_cast<volatile int *>(smem + L::kOffMeta + kMetaJ);
    volatile int *meta_f = reinterpret_cast<volatile int *>(smem + L::kOffMeta + kMetaF);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kOffMeta + kAbortFlag);
    const uint32_t bar_tile = meta + kBarTile, bar_fin = meta + kBarFin;
#define BAR_K_FULL(s) (meta + kBarFull + 8u * (uint32_t)(s))
#define BAR_K_EMPTY(s) (meta + kBarEmpty + 8u * (uint32_t)(s))
#define BAR_V_FULL(s) (meta + kBarVFull + 8u * (uint32_t)(s))
#define BAR_V_EMPTY(s) (meta + kBarVEmpty + 8u * (uint32_t)(s))
#define BAR_S_FULL(b) (meta + kBarSFull + 8u * (uint32_t)(b))
#define BAR_P_FULL(b) (meta + kBarPFull + 8u * (uint32_t)(b))
#define BAR_DONE(b) (meta + kBarDone + 8u * (uint32_t)(b))

    const int tid = threadIdx.x, warp = tid >> 5;
    const int lane_id = blockIdx.x;
    const int tile = (int)gridDim.y - 1 - (int)blockIdx.y;  // two query blocks
    const int qa = 2 * tile;                                 // longest rows first
    const bool has_b = qa + 1 < nb;
    constexpr uint32_t kAcc = kDiff ? kDiffAccCol : kAccCol;

    // The first global reads are issued together and waited for at the barrier below: whether
    // the launch already gave up elsewhere (one thread, so the whole CTA takes the same branch),
    // and the producer's two CSR rows.
    const bool gave_up = tid == 0 && *reinterpret_cast<volatile unsigned *>(flags.abort_epoch) == flags.epoch;
    ListUnion lu;
    if (warp == kProducerWarp && elect_one()) {
        lu.a = col_idx + row_ptr[qa];
        lu.ia = 0;
        lu.ia_end = vlen[qa];
        lu.b = has_b ? col_idx + row_ptr[qa + 1] : col_idx;
        lu.ib = 0;
        lu.ib_end = has_b ? vlen[qa + 1] : 0;
    }

    if (tid == 0) {
        mbar_init(bar_tile, 1);
        for (int s = 0; s < kStream; ++s) {
            mbar_init(BAR_K_FULL(s), 1);
            mbar_init(BAR_K_EMPTY(s), 1);
            mbar_init(BAR_V_FULL(s), 1);
            mbar_init(BAR_V_EMPTY(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(BAR_S_FULL(b), 1);
            mbar_init(BAR_P_FULL(b), kElt);
            mbar_init(BAR_DONE(b), 1);
        }
        mbar_init(bar_fin, 1);
        *abort_flag = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(meta + kTmemSlot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    const bool leave = __syncthreads_or(gave_up);
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::kOffMeta + kTmemSlot);
    if (leave) {  // nothing was issued yet: give the columns back and go
        if (tid == 0) raise_status(flags, kDevTimeout);  // a replayed launch that gave up once says so again
        if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
        return;
    }

    if (warp == kProducerWarp) {
        if (elect_one()) {
            tma_prefetch_desc(&tmQ);
            tma_prefetch_desc(&tmdO);
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
            tma_prefetch_desc(&tmdQ);
            mbar_arrive_expect_tx(bar_tile, 2 * L::kTileBytes);
#pragma unroll
            for (int c = 0; c < L::kChunks; ++c) {
                tma_load_3d(sQ + c * 16384, &tmQ, c * 64, qa * kBlock, lane_id, bar_tile);
                tma_load_3d(sdO + c * 16384, &tmdO, c * 64, qa * kBlock, lane_id, bar_tile);
            }
            bool ok = true;
            int k_issued = 0, v_issued = 0;
            for (int v = 0;; ++v) {
                const int s = v % kStream;
                const uint32_t par = (uint32_t)((v / kStream) - 1) & 1u;
                if (v >= kStream && !mbar_wait(BAR_K_EMPTY(s), par, flags)) { ok = false; break; }
                int f = 0;
                const int j = lu.next(f);
                meta_j[v % kMetaRing] = j;
                meta_f[v % kMetaRing] = f;
                if (j < 0) {
                    mbar_arrive(BAR_K_FULL(s));
                    break;
                }
                mbar_arrive_expect_tx(BAR_K_FULL(s), L::kKVBytes);
#pragma unroll
                for (int c = 0; c < L::kChunks; ++c)
                    tma_load_3d(sK + s * L::kKVBytes + c * 8192, &tmK, c * 64, j * kBlock, lane_id,
                                     BAR_K_FULL(s));
                k_issued = v + 1;
                if (v >= kStream && !mbar_wait(BAR_V_EMPTY(s), par, flags)) { ok = false; break; }
                mbar_arrive_expect_tx(BAR_V_FULL(s), L::kKVBytes);
#pragma unroll
                for (int c = 0; c < L::kChunks; ++c)
                    tma_load_3d(sV + s * L::kKVBytes + c * 8192, &tmV, c * 64, j * kBlock, lane_id,
                                     BAR_V_FULL(s));
                v_issued = v + 1;
            }
            if (!ok) {
                *abort_flag = 1;
                (void)mbar_wait_timed(bar_tile, 0);
                for (int w = k_issued - kStream; w < k_issued; ++w)
                    if (w >= 0) (void)mbar_wait_timed(BAR_K_FULL(w % kStream), (w / kStream) & 1);
                for (int w = v_issued - kStream; w < v_issued; ++w)
                    if (w >= 0) (void)mbar_wait_timed(BAR_V_FULL(w % kStream), (w / kStream) & 1);
            }
        }
    } else if (warp == kMmaWarp) {
        if (elect_one()) {
            constexpr uint32_t kIdescS = idesc_f16(kBF16, 128, 64, false);
            constexpr uint32_t kIdescAcc = idesc_f16(kBF16, 128, kDiff ? D / 2 : D, true);
            const uint64_t q_desc = sdesc_sw128(sQ, 16, 1024), do_desc = sdesc_sw128(sdO, 16, 1024),
                           k_desc = sdesc_sw128(sK, 16, 1024), v_desc = sdesc_sw128(sV, 16, 1024),
                           kt_desc = sdesc_sw128(sK, 8192, 1024);
            bool ok = mbar_wait(bar_tile, 0, flags);
            int u = 0;
            bool have = false;
            // products of step uu: S = Q K^T and dP = dO V^T; V's stage is free afterwards
            auto issue_products = [&](int uu) -> bool {
                const int s_ = uu % kStream;
                if (!mbar_wait(BAR_V_FULL(s_), (uu / kStream) & 1, flags)) return false;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t aoff = (kk >> 2) * 16384 + (kk & 3) * 32;
                    const uint32_t boff = s_ * L::kKVBytes + (kk >> 2) * 8192 + (kk & 3) * 32;
                    const bool second = kDiff && kk >= D / 32;  // the second map's half of the columns
                    tc_mma_ss(tmem + (second ? s2_col(uu & 1) : s_col(uu & 1)), sdesc_at(q_desc, aoff),
                              sdesc_at(k_desc, boff), kIdescS, kk % (kDiff ? D / 32 : D / 16) > 0 ? 1u : 0u);
                }
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t aoff = (kk >> 2) * 16384 + (kk & 3) * 32;
                    const uint32_t boff = s_ * L::kKVBytes + (kk >> 2) * 8192 + (kk & 3) * 32;
                    tc_mma_ss(tmem + (kDiff ? diff_dp_col(uu & 1) : dp_col(uu & 1)), sdesc_at(do_desc, aoff),
                              sdesc_at(v_desc, boff), kIdescS, kk > 0 ? 1u : 0u);
                }
                tc_commit(BAR_S_FULL(uu & 1));
                tc_commit(BAR_V_EMPTY(s_));
                return true;
            };
            if (ok) {
                ok = mbar_wait(BAR_K_FULL(0), 0, flags);
                if (ok) {
                    if (meta_j[0] >= 0) {
                        ok = issue_products(0);
                        have = ok;
                    } else {
                        mbar_arrive(BAR_S_FULL(0));
                    }
                }
            }
            while (ok && have) {
                bool next = false;
                const int s1 = (u + 1) % kStream;
                ok = mbar_wait(BAR_K_FULL(s1), ((u + 1) / kStream) & 1, flags);
                if (!ok) break;
                if (meta_j[(u + 1) % kMetaRing] >= 0) {
                    ok = issue_products(u + 1);
                    if (!ok) break;
                    next = true;
                } else {
                    mbar_arrive(BAR_S_FULL((u + 1) & 1));
                }
                // dQ += dS_u K_u once the elementwise warps have written dS_u
                ok = mbar_wait(BAR_P_FULL(u & 1), (u >> 1) & 1, flags);
                if (!ok) break;
                const int s = u % kStream;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    tc_mma_ts(tmem + kAcc, tmem + s_col(u & 1) + packed_col(kk),
                              sdesc_at(kt_desc, s * L::kKVBytes + kk * 2048), kIdescAcc,
                              (u > 0 || kk > 0) ? 1u : 0u);
                if constexpr (kDiff) {  // dS2 with the second half of K's columns
                    constexpr uint32_t kHalf = D == 128 ? 8192 : 64;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc_mma_ts(tmem + kAcc + D / 2, tmem + s2_col(u & 1) + packed_col(kk),
                                  sdesc_at(kt_desc, s * L::kKVBytes + kk * 2048 + kHalf), kIdescAcc,
                                  (u > 0 || kk > 0) ? 1u : 0u);
                }
                tc_commit(BAR_K_EMPTY(s));
                tc_commit(BAR_DONE(u & 1));
                have = next;
                ++u;
            }
            if (!ok) *abort_flag = 1;
            tc_commit(bar_fin);
            (void)mbar_wait_timed(bar_fin, 0);
        }
    } else {
        // ------------------------------------------------------------ elementwise (warps 0-7)
        const int row = tid & 127, col0 = (tid >> 7) * 32;  // this thread's row, and first column of a step
        const int half = row >> 6;
        const int r_in = row & 63;
        const int my_block = qa + half;
        const bool row_exists = half == 0 || has_b;
        const uint32_t t_lane = (uint32_t)((warp & 3) * 32) << 16;
        // the row in the per-lane padded Delta / log-sum-exp arrays (nb * 64 rows per lane)
        const long long grow = ((long long)lane_id * nb + qa) * kBlock + row;
        const float lse2 = row_exists ? lse[grow] : INFINITY;
        const float dlt = row_exists ? delta[grow] : 0.f;
        bool ok = true;
        // kDiff: the second map, whose dP is -lambda dO V^T
        [[maybe_unused]] float lse2_b = INFINITY, dlt_b = 0.f, mul = 0.f;
        [[maybe_unused]] float dot[2] = {0.f, 0.f};  // the sum of P2 o dO V^T over the row
        if constexpr (kDiff) {
            mul = -lambda_of<D / 2, kBF16>(terms, lane_id % terms.H);
            if (row_exists) {
                lse2_b = lse[terms.map_rows + grow];
                dlt_b = delta[terms.map_rows + grow] * mul;
            }
        }
        // kBias: the sum over the row of the dS that lie before the last bucket
        [[maybe_unused]] float others = 0.f, last_bias = 0.f;
        [[maybe_unused]] uint32_t reached = 0u;  // the bits of the last bucket's dS: their sign aside 0 if all of them are 0
        [[maybe_unused]] float *win = reinterpret_cast<float *>(smem + L::kOffWin) + warp * kWindow;
        [[maybe_unused]] float *bins = reinterpret_cast<float *>(smem + L::kOffBins) + warp * kMaxBuckets;
        [[maybe_unused]] float *near_sums =
            reinterpret_cast<float *>(smem + L::kOffNear) + warp * kNearRow + kDistFront;
        [[maybe_unused]] const int wlane = tid & 31;
        [[maybe_unused]] int known = 0;  // distances in the table
        [[maybe_unused]] int last_bucket = 0, last_start = 0;
        if constexpr (kBias) {
            for (int b = wlane; b < kMaxBuckets; b += 32) bins[b] = 0.f;
            for (int d = wlane - kDistFront; d < kNearRow - kDistFront; d += 32) near_sums[d] = 0.f;
            table.template load<kBF16>(terms, lane_id % terms.H, tid, kElt);
            named_barrier(2, kElt);
            last_bucket = terms.n - 1;
            last_start = table.start[last_bucket];
            last_bias = table.bias[last_bucket];
            known = table.spread(terms.n, (qa + 2) * kBlock, tid, kElt);
            named_barrier(2, kElt);
        }
        int u = 0;
        for (; ok; ++u) {
            // (all lanes together: one whose wait ran out must not leave the others to a warp-wide step)
            const bool there = mbar_wait(BAR_S_FULL(u & 1), (u >> 1) & 1, flags);
            if (!__all_sync(0xffffffffu, there)) { ok = false; break; }
            const int j = meta_j[u % kMetaRing];
            const int fl = meta_f[u % kMetaRing];
            if (j < 0) break;
            tc_fence_after();
            const bool in_row = row_exists && ((fl >> half) & 1);  // warp-uniform
            const uint32_t s_at = tmem + t_lane + s_col(u & 1) + col0;
            const uint32_t dp_at = tmem + t_lane + (kDiff ? diff_dp_col(u & 1) : dp_col(u & 1)) + col0;
            [[maybe_unused]] const uint32_t s2_at = tmem + t_lane + s2_col(u & 1) + col0;
            uint32_t dsw[16];
            [[maybe_unused]] uint32_t dsw2[16];
            __syncwarp();
            if (in_row) {
                // the bias: one constant for the step, or a window (key c at distance d_lo + 63 + wlane - c)
                [[maybe_unused]] bool near = false;
                [[maybe_unused]] int d_lo = 0, d_hi = 0;
                float zero_at = -lse2;
                if constexpr (kBias) {
                    d_lo = (qa - j) * kBlock + (warp & 3) * 32 - 63;
                    d_hi = d_lo + kWindow - 2;
                    near = last_start > d_lo || j == my_block;
                    if (!near) zero_at += last_bias;
                }
                if (!near) {
                    const bool diagonal = !kBias && j == my_block;
                    const float delta_at = dlt;
                    [[maybe_unused]] const float zero_b = -lse2_b, delta_b = dlt_b, times = mul;
                    auto step = [&, zero_at, delta_at, zero_b, delta_b, times](auto is_diagonal) {
                        constexpr bool kDiagonal = decltype(is_diagonal)::value;
                        uint32_t sr[32], pr[32];
                        [[maybe_unused]] uint32_t sr2[32];
                        if constexpr (kDiff) tmem_ld32_three(s_at, sr, s2_at, sr2, dp_at, pr);
                        else tmem_ld32_pair(s_at, sr, dp_at, pr);
#pragma unroll
                        for (int t = 0; t < 16; ++t) {
                            float ds[2];
                            [[maybe_unused]] float ds2[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float s = __uint_as_float(sr[2 * t + e]), dp = __uint_as_float(pr[2 * t + e]);
                                float p = ex2_approx(fmaf(s, scale_log2, zero_at));
                                if constexpr (kDiagonal) p = 2 * t + e > r_in - col0 ? 0.f : p;
                                ds[e] = p * (dp - delta_at);
                                if constexpr (kDiff) {
                                    float p2 = ex2_approx(fmaf(__uint_as_float(sr2[2 * t + e]), scale_log2, zero_b));
                                    if constexpr (kDiagonal) p2 = 2 * t + e > r_in - col0 ? 0.f : p2;
                                    ds2[e] = p2 * fmaf(dp, times, -delta_b);
                                    dot[e] = fmaf(p2, dp, dot[e]);
                                }
                            }
                            dsw[t] = pack16x2<kBF16>(ds[0], ds[1]);
                            if constexpr (kDiff) dsw2[t] = pack16x2<kBF16>(ds2[0], ds2[1]);
                        }
                    };
                    if (diagonal) step(std::true_type{});  // a loop of its own
                    else step(std::false_type{});
                    if constexpr (kBias) {
#pragma unroll
                        for (int t = 0; t < 16; ++t) reached |= dsw[t];
                    }
                } else if constexpr (kBias) {
                    const float *wp = window_at(win, table, known, terms.n, d_lo, wlane) + 63 + wlane - col0;
                    // columns up to this one lie in the last bucket
                    const int far_to = d_lo + 63 + wlane - col0 - last_start;
                    uint32_t sr[32], pr[32];
                    tmem_ld32_pair(s_at, sr, dp_at, pr);
                    float x[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) x[c] = fmaf(__uint_as_float(sr[c]), scale_log2, wp[-c]) + zero_at;
                    if (j == my_block) {
#pragma unroll
                        for (int c = 0; c < 32; ++c) x[c] = c > r_in - col0 ? -INFINITY : x[c];
                    }
#pragma unroll
                    for (int c = 0; c < 32; ++c) x[c] = ex2_approx(x[c]) * (__uint_as_float(pr[c]) - dlt);
#pragma unroll
                    for (int t = 0; t < 16; ++t) dsw[t] = pack16x2<kBF16>(x[2 * t], x[2 * t + 1]);
                    // the sum over the row, without the last bucket's keys
                    if (d_hi < last_start) {
                        uint64_t two[4];
#pragma unroll
                        for (int t = 0; t < 4; ++t) two[t] = f2_pack(x[2 * t], x[2 * t + 1]);
#pragma unroll
                        for (int t = 4; t < 16; ++t) two[t & 3] = f2_add(two[t & 3], f2_pack(x[2 * t], x[2 * t + 1]));
                        float s0, s1;
                        f2_unpack(f2_add(f2_add(two[0], two[1]), f2_add(two[2], two[3])), s0, s1);
                        others += s0 + s1;
                    } else {
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            others += c > far_to ? x[c] : 0.f;
                            reached |= c <= far_to && x[c] != 0.f ? 1u : 0u;
                        }
                    }
                    // the sums over the diagonals: column c of row (lane + c + 1) mod 32 lies at the distance
                    // d_lo + 64 - col0 + lane, or 32 nearer once the row wraps
                    float below = 0.f, above = 0.f;
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const float y = __shfl_sync(0xffffffffu, x[c], (wlane + c + 1) & 31);
                        const bool first = wlane + c + 1 < 32;
                        below += first ? y : 0.f;
                        above += first ? 0.f : y;
                    }
                    __syncwarp();  // the window has been read
                    if (d_hi < kNearSums) {
                        float *to = near_sums + d_lo + 32 - col0 + wlane;
                        to[32] += below;
                        to[0] += above;
                    } else {
                        const bool second = col0 > 0;
                        add_distances(bins, win, second ? above : 0.f, second ? below : above, second ? 0.f : below, table,
                                      table.find(terms.n, d_hi), last_bucket, d_lo, d_hi, wlane);
                    }
                }
            } else {
#pragma unroll
                for (int t = 0; t < 16; ++t) {
                    dsw[t] = 0u;
                    if constexpr (kDiff) dsw2[t] = 0u;
                }
            }
            __syncwarp();
            tmem_st16(s_at, dsw);  // dS_u over the first 16 of this warp's columns of S_u
            if constexpr (kDiff) tmem_st16(s2_at, dsw2);
            tc_fence_before();
            mbar_arrive(BAR_P_FULL(u & 1));
        }
        if (!ok) *abort_flag = 1;
        bool acc_valid = false;
        if (ok && u > 0) {
            // the last two steps' accumulations: those before had completed when the last step's
            // products did
            acc_valid = mbar_wait(BAR_DONE((u - 1) & 1), ((u - 1) >> 1) & 1, flags) &&
                        (u < 2 || mbar_wait(BAR_DONE(u & 1), ((u - 2) >> 1) & 1, flags));
            if (!acc_valid) *abort_flag = 1;
        }
        if constexpr (kBias) {  // for the warp with the row's other columns; the window has been read
            __syncwarp();
            win[wlane] = __uint_as_float(reached);
        }
        // one decision for all elementwise warps (the section below has a barrier of its own)
        if (!named_barrier_or(1, kElt, *abort_flag != 0)) {
            tc_fence_after();
            __syncwarp();
            // every product that read Q has completed: Q's tile stages dQ
            stage_rows<D, kBF16>(tmem + t_lane, kAcc, acc_valid, scale, sQ, row, tid >> 7);
            if constexpr (kBias) {
                // the last bucket, unless none of its keys has any weight in the row
                reached |= __float_as_uint(win[((warp ^ 4) - warp) * kWindow + wlane]);
                float s = (reached & 0x7FFF7FFFu) != 0u ? -others : 0.f;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                if (wlane == 0) bins[last_bucket] = s;
            }
            if constexpr (kDiff) {
                float s = dot[0] + dot[1];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                if (wlane == 0) reinterpret_cast<float *>(smem + L::kOffDO)[warp] = s;  // dO's tile is free as well
            }
            fence_proxy_async_smem();
            named_barrier(1, kElt);
            if constexpr (kBias) {
                // the warps' bucket sums and their sums by distance, a thread per bucket
                const float *all = reinterpret_cast<const float *>(smem + L::kOffBins);
                const float *by = reinterpret_cast<const float *>(smem + L::kOffNear) + kDistFront;
                float *to = partial + ((long long)lane_id * gridDim.y + tile) * terms.n;
                for (int b = tid; b < terms.n; b += kElt) {
                    float s = 0.f;
#pragma unroll
                    for (int w = 0; w < kEltWarps; ++w) s += all[w * kMaxBuckets + b];
                    const int end = b < last_bucket ? min(table.start[b + 1], kNearSums) : 0;
                    for (int d = table.start[b]; d < end; ++d)
#pragma unroll
                        for (int w = 0; w < kEltWarps; ++w) s += by[w * kNearRow + d];
                    to[b] = s;
                }
            }
            if constexpr (kDiff) {
                const float *by = reinterpret_cast<const float *>(smem + L::kOffDO);
                if (tid == 0) {
                    float s = 0.f;
#pragma unroll
                    for (int w = 0; w < kEltWarps; ++w) s += by[w];
                    partial[(long long)lane_id * gridDim.y + tile] = -s;
                }
            }
            if (tid == 0) {
#pragma unroll
                for (int c = 0; c < L::kChunks; ++c) {
                    tma_store_3d(&tmdQ, c * 64, qa * kBlock, lane_id, sQ + c * 16384);
                    if (has_b) tma_store_3d(&tmdQ, c * 64, (qa + 1) * kBlock, lane_id, sQ + c * 16384 + 8192);
                }
                tma_store_commit();
                tma_store_wait_read();
            }
        }
    }
#undef BAR_K_FULL
#undef BAR_K_EMPTY
#undef BAR_V_FULL
#undef BAR_V_EMPTY
#undef BAR_S_FULL
#undef BAR_P_FULL
#undef BAR_DONE
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) {
        raise_status(flags, kDevTimeout);
        atomicExch(flags.abort_epoch, flags.epoch);
    }
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ---------------------------------------------------------------- dK, dV
template <int D, class Terms>
struct DkvSmem {
    static constexpr int kRowBytes = Terms::kDiff ? 512 : 256;  // a step's 64 floats, of each map
    static constexpr int kChunks = D / 64;
    static constexpr int kTileBytes = kRows * D * 2;   // K and V tiles (128 keys)
    static constexpr int kQBytes = kBlock * D * 2;     // one Q or dO block
    static constexpr int kOffK = 0;
    static constexpr int kOffV = kOffK + kTileBytes;
    static constexpr int kRing = Terms::kDiff && D == 128 ? 3 : kStream;  // two tiles of P beside it
    static constexpr int kOffQ = kOffV + kTileBytes;
    static constexpr int kOffDO = kOffQ + kRing * kQBytes;
    static constexpr int kOffP = kOffDO + kRing * kQBytes;          // kDiff: P1 - lambda P2 of two steps, transposed
    static constexpr int kPBytes = kRows * kBlock * 2;
    static constexpr int kOffLse = kOffP + (Terms::kDiff ? 2 * kPBytes : 0);  // kRing x 64 floats (kDiff: of each map)
    static constexpr int kOffDelta = kOffLse + kRing * kRowBytes;
    static constexpr int kOffMeta = kOffDelta + kRing * kRowBytes;
    static constexpr int kOffTable = kOffMeta + kMetaBytes;        // bias only
    static constexpr int kOffWin = kOffTable + kBucketTableBytes;  // a window of each warp (bias only)
    static constexpr int kEnd = Terms::kBias ? kOffWin + kEltWarps * kWindow * 4 : kOffTable;
    static constexpr int kBytes = smem_bytes_one_cta(kEnd + 1024);
};

template <int D, bool kBF16, class Terms>
__global__ void __launch_bounds__(kThreads, 1)
bwd_dkv_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
               const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmdO,
               const __grid_constant__ CUtensorMap tmdK, const __grid_constant__ CUtensorMap tmdV,
               const int *__restrict__ col_ptr, const int32_t *__restrict__ row_idx,
               const int *__restrict__ pairs, const float *__restrict__ lse,
               const float *__restrict__ delta, int nb, int S, float scale, float scale_log2,
               DeviceFlags flags, const __grid_constant__ Terms terms) {
    constexpr bool kBias = Terms::kBias, kDiff = Terms::kDiff;
    using L = DkvSmem<D, Terms>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_base = smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    if (base - raw_base + L::kEnd > (uint32_t)L::kBytes) {
        if (threadIdx.x == 0) raise_status(flags, kDevSmemAlign);
        return;
    }
    uint8_t *smem = smem_raw + (base - raw_base);
    [[maybe_unused]] const BucketTable table(smem + L::kOffTable);
    const uint32_t sK = base + L::kOffK, sV = base + L::kOffV, sQ = base + L::kOffQ, sdO = base + L::kOffDO;
    [[maybe_unused]] const uint32_t sP = base + L::kOffP;
    const uint32_t sLse = base + L::kOffLse, sDelta = base + L::kOffDelta;
    const float *lse_s = reinterpret_cast<const float *>(smem + L::kOffLse);
    const float *delta_s = reinterpret_cast<const float *>(smem + L::kOffDelta);
    const uint32_t meta = base + L::kOffMeta;
    volatile int *meta_j = reinterpret_cast<volatile int *>(smem + L::kOffMeta + kMetaJ);
    volatile int *meta_f = reinterpret_cast<volatile int *>(smem + L::kOffMeta + kMetaF);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kOffMeta + kAbortFlag);
    const uint32_t bar_tile = meta + kBarTile, bar_fin = meta + kBarFin;
#define BAR_FULL(s) (meta + kBarFull + 8u * (uint32_t)(s))
#define BAR_EMPTY(s) (meta + kBarEmpty + 8u * (uint32_t)(s))
#define BAR_S_FULL(b) (meta + kBarSFull + 8u * (uint32_t)(b))
#define BAR_P_FULL(b) (meta + kBarPFull + 8u * (uint32_t)(b))
#define BAR_DONE(b) (meta + kBarDone + 8u * (uint32_t)(b))
#define BAR_LOADED(b) (meta + kBarLoaded + 8u * (uint32_t)(b))

    const int tid = threadIdx.x, warp = tid >> 5;
    const int lane_id = blockIdx.x;
    // key blocks ka and kb (-1: none) from the pair list, heaviest transposed columns first
    const int ka = __ldg(pairs + 2 * blockIdx.y), kb = __ldg(pairs + 2 * blockIdx.y + 1);
    const bool has_b = kb >= 0;

    // As in the dQ kernel: the abort flag and the producer's two transposed columns are read
    // before the first barrier.
    const bool gave_up = tid == 0 && *reinterpret_cast<volatile unsigned *>(flags.abort_epoch) == flags.epoch;
    ListUnion lu;
    if (warp == kProducerWarp && elect_one()) {
        lu.a = row_idx + col_ptr[ka];
        lu.ia = 0;
        lu.ia_end = col_ptr[ka + 1] - col_ptr[ka];
        lu.b = has_b ? row_idx + col_ptr[kb] : row_idx;
        lu.ib = 0;
        lu.ib_end = has_b ? col_ptr[kb + 1] - col_ptr[kb] : 0;
    }

    if (tid == 0) {
        mbar_init(bar_tile, 1);
        for (int s = 0; s < L::kRing; ++s) {
            mbar_init(BAR_FULL(s), 1);
            mbar_init(BAR_EMPTY(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(BAR_S_FULL(b), 1);
            mbar_init(BAR_P_FULL(b), kElt);
            mbar_init(BAR_DONE(b), 1);
        }
        mbar_init(bar_fin, 1);
        if constexpr (kDiff)
            for (int b = 0; b < 2; ++b) mbar_init(BAR_LOADED(b), kElt);
        *abort_flag = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(meta + kTmemSlot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    const bool leave = __syncthreads_or(gave_up);
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::kOffMeta + kTmemSlot);
    if (leave) {  // nothing was issued yet: give the columns back and go
        if (tid == 0) raise_status(flags, kDevTimeout);  // a replayed launch that gave up once says so again
        if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
        return;
    }
    constexpr uint32_t kDVCol = kAccCol, kDKCol = kAccCol + D;

    if (warp == kProducerWarp) {
        if (elect_one()) {
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
            tma_prefetch_desc(&tmQ);
            tma_prefetch_desc(&tmdO);
            tma_prefetch_desc(&tmdK);
            tma_prefetch_desc(&tmdV);
            mbar_arrive_expect_tx(bar_tile, 2 * L::kTileBytes);
#pragma unroll
            for (int c = 0; c < L::kChunks; ++c) {
                tma_load_3d(sK + c * 16384, &tmK, c * 64, ka * kBlock, lane_id, bar_tile);
                tma_load_3d(sV + c * 16384, &tmV, c * 64, ka * kBlock, lane_id, bar_tile);
                // the second block's rows, or the first block's again (masked) if there is none
                const int y2 = (has_b ? kb : ka) * kBlock;
                tma_load_3d(sK + c * 16384 + 8192, &tmK, c * 64, y2, lane_id, bar_tile);
                tma_load_3d(sV + c * 16384 + 8192, &tmV, c * 64, y2, lane_id, bar_tile);
            }
            bool ok = true;
            int issued = 0;
            for (int v = 0;; ++v) {
                const int s = v % L::kRing;
                const uint32_t par = (uint32_t)((v / L::kRing) - 1) & 1u;
                if (v >= L::kRing && !mbar_wait(BAR_EMPTY(s), par, flags)) { ok = false; break; }
                int f = 0;
                const int i = lu.next(f);
                meta_j[v % kMetaRing] = i;
                meta_f[v % kMetaRing] = f;
                if (i < 0) {
                    mbar_arrive(BAR_FULL(s));
                    break;
                }
                mbar_arrive_expect_tx(BAR_FULL(s), 2 * L::kQBytes + 2 * L::kRowBytes);
#pragma unroll
                for (int c = 0; c < L::kChunks; ++c) {
                    tma_load_3d(sQ + s * L::kQBytes + c * 8192, &tmQ, c * 64, i * kBlock, lane_id, BAR_FULL(s));
                    tma_load_3d(sdO + s * L::kQBytes + c * 8192, &tmdO, c * 64, i * kBlock, lane_id, BAR_FULL(s));
                }
                const long long py = ((long long)lane_id * nb + i) * kBlock;  // padded row
                bulk_load(sLse + s * L::kRowBytes, lse + py, 256, BAR_FULL(s));
                bulk_load(sDelta + s * L::kRowBytes, delta + py, 256, BAR_FULL(s));
                if constexpr (kDiff) {
                    bulk_load(sLse + s * L::kRowBytes + 256, lse + terms.map_rows + py, 256, BAR_FULL(s));
                    bulk_load(sDelta + s * L::kRowBytes + 256, delta + terms.map_rows + py, 256, BAR_FULL(s));
                }
                issued = v + 1;
            }
            if (!ok) {
                *abort_flag = 1;
                (void)mbar_wait_timed(bar_tile, 0);
                for (int w = issued - L::kRing; w < issued; ++w)
                    if (w >= 0) (void)mbar_wait_timed(BAR_FULL(w % L::kRing), (w / L::kRing) & 1);
            }
        }
    } else if (warp == kMmaWarp) {
        if (elect_one()) {
            constexpr uint32_t kIdescS = idesc_f16(kBF16, 128, 64, false);
            constexpr uint32_t kIdescAcc = idesc_f16(kBF16, 128, D, true);
            const uint64_t k_desc = sdesc_sw128(sK, 16, 1024), v_desc = sdesc_sw128(sV, 16, 1024),
                           q_desc = sdesc_sw128(sQ, 16, 1024), do_desc = sdesc_sw128(sdO, 16, 1024),
                           qt_desc = sdesc_sw128(sQ, 8192, 1024), dot_desc = sdesc_sw128(sdO, 8192, 1024);
            bool ok = mbar_wait(bar_tile, 0, flags);
            if constexpr (kDiff) {
                // Step u's three products go to the slots 3u, 3u + 1, 3u + 2 (mod 4) of 64 columns, S1^T, S2^T,
                // dP^T; its dS1^T and dS2^T come back in the third, P^T in shared memory.  So S1 of the next
                // step has a slot of its own, and S2 and dP can follow as soon as this step's scores are read.
                constexpr uint32_t kIdescHalf = idesc_f16(kBF16, 128, D / 2, true);
                constexpr uint32_t kHalf = D == 128 ? 8192 : 64;  // the second half of Q's columns
                const uint64_t p_desc = sdesc_sw128(sP, 16, 1024);
                auto issue = [&](int uu, int x) {  // product x of step uu
                    const int s_ = uu % L::kRing;
                    const uint32_t to = tmem + diff_slot(uu, x);
                    if (x < 2) {
#pragma unroll
                        for (int k = 0; k < D / 32; ++k) {
                            const int kk = k + x * (D / 32);
                            tc_mma_ss(to, sdesc_at(k_desc, (kk >> 2) * 16384 + (kk & 3) * 32),
                                      sdesc_at(q_desc, s_ * L::kQBytes + (kk >> 2) * 8192 + (kk & 3) * 32), kIdescS,
                                      k > 0 ? 1u : 0u);
                        }
                    } else {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            tc_mma_ss(to, sdesc_at(v_desc, (kk >> 2) * 16384 + (kk & 3) * 32),
                                      sdesc_at(do_desc, s_ * L::kQBytes + (kk >> 2) * 8192 + (kk & 3) * 32), kIdescS,
                                      kk > 0 ? 1u : 0u);
                    }
                };
                ok = ok && mbar_wait(BAR_FULL(0), 0, flags);
                bool have = false;
                if (ok) {
                    have = meta_j[0] >= 0;
                    if (have) {
                        tc_fence_after();
                        issue(0, 0);
                        issue(0, 1);
                        issue(0, 2);
                        tc_commit(BAR_S_FULL(0));
                    } else {
                        mbar_arrive(BAR_S_FULL(0));
                    }
                }
                for (int u = 0; ok && have; ++u) {
                    const int s = u % L::kRing, b = u & 1, s1 = (u + 1) % L::kRing;
                    ok = mbar_wait(BAR_FULL(s1), ((u + 1) / L::kRing) & 1, flags);
                    if (!ok) break;
                    const bool next = meta_j[(u + 1) % kMetaRing] >= 0;
                    if (next) {
                        tc_fence_after();
                        issue(u + 1, 0);
                    }
                    ok = mbar_wait(BAR_LOADED(b), (u >> 1) & 1, flags);
                    if (!ok) break;
                    if (next) {
                        tc_fence_after();
                        issue(u + 1, 1);
                        issue(u + 1, 2);
                        tc_commit(BAR_S_FULL(b ^ 1));
                    } else {
                        mbar_arrive(BAR_S_FULL(b ^ 1));
                    }
                    ok = mbar_wait(BAR_P_FULL(b), (u >> 1) & 1, flags);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc_mma_ss(tmem + kDVCol, sdesc_at(p_desc, b * L::kPBytes + kk * 32),
                                  sdesc_at(dot_desc, s * L::kQBytes + kk * 2048), kIdescAcc, (u > 0 || kk > 0) ? 1u : 0u);
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            tc_mma_ts(tmem + kDKCol + m * (D / 2), tmem + diff_slot(u, 2) + m * 16 + packed_col(kk),
                                      sdesc_at(qt_desc, s * L::kQBytes + kk * 2048 + m * kHalf), kIdescHalf,
                                      (u > 0 || kk > 0) ? 1u : 0u);
                    tc_commit(BAR_EMPTY(s));
                    tc_commit(BAR_DONE(b));
                    have = next;
                }
            } else {
                int u = 0;
                bool have = false;
                // products of step uu: S^T = K Q^T and dP^T = V dO^T
                auto issue_products = [&](int uu) {
                    const int s_ = uu % L::kRing;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t aoff = (kk >> 2) * 16384 + (kk & 3) * 32;
                        const uint32_t boff = s_ * L::kQBytes + (kk >> 2) * 8192 + (kk & 3) * 32;
                        tc_mma_ss(tmem + s_col(uu & 1), sdesc_at(k_desc, aoff), sdesc_at(q_desc, boff),
                                  kIdescS, kk > 0 ? 1u : 0u);
                    }
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t aoff = (kk >> 2) * 16384 + (kk & 3) * 32;
                        const uint32_t boff = s_ * L::kQBytes + (kk >> 2) * 8192 + (kk & 3) * 32;
                        tc_mma_ss(tmem + dp_col(uu & 1), sdesc_at(v_desc, aoff), sdesc_at(do_desc, boff),
                                  kIdescS, kk > 0 ? 1u : 0u);
                    }
                    tc_commit(BAR_S_FULL(uu & 1));
                };
                if (ok) {
                    ok = mbar_wait(BAR_FULL(0), 0, flags);
                    if (ok) {
                        if (meta_j[0] >= 0) {
                            issue_products(0);
                            have = true;
                        } else {
                            mbar_arrive(BAR_S_FULL(0));
                        }
                    }
                }
                while (ok && have) {
                    bool next = false;
                    const int s1 = (u + 1) % L::kRing;
                    ok = mbar_wait(BAR_FULL(s1), ((u + 1) / L::kRing) & 1, flags);
                    if (!ok) break;
                    if (meta_j[(u + 1) % kMetaRing] >= 0) {
                        issue_products(u + 1);
                        next = true;
                    } else {
                        mbar_arrive(BAR_S_FULL((u + 1) & 1));
                    }
                    // dV += P^T_u dO_u and dK += dS^T_u Q_u once the elementwise warps wrote them
                    ok = mbar_wait(BAR_P_FULL(u & 1), (u >> 1) & 1, flags);
                    if (!ok) break;
                    const int s = u % L::kRing;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc_mma_ts(tmem + kDVCol, tmem + s_col(u & 1) + packed_col(kk),
                                  sdesc_at(dot_desc, s * L::kQBytes + kk * 2048), kIdescAcc,
                                  (u > 0 || kk > 0) ? 1u : 0u);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        tc_mma_ts(tmem + kDKCol, tmem + dp_col(u & 1) + packed_col(kk),
                                  sdesc_at(qt_desc, s * L::kQBytes + kk * 2048), kIdescAcc,
                                  (u > 0 || kk > 0) ? 1u : 0u);
                    tc_commit(BAR_EMPTY(s));
                    tc_commit(BAR_DONE(u & 1));
                    have = next;
                    ++u;
                }
            }
            if (!ok) *abort_flag = 1;
            tc_commit(bar_fin);
            (void)mbar_wait_timed(bar_fin, 0);
        }
    } else {
        // ------------------------------------------------------------ elementwise (warps 0-7)
        const int row = tid & 127, col0 = (tid >> 7) * 32;  // this thread's row, and first column of a step
        const int half = row >> 6;               // 0: key block ka, 1: key block kb
        const int k_in = row & 63;               // key token within its block
        const int key_block = half ? kb : ka;
        const bool row_exists = half == 0 || has_b;
        const uint32_t t_lane = (uint32_t)((warp & 3) * 32) << 16;
        bool ok = true;
        [[maybe_unused]] float mul = 0.f;  // kDiff: the second map's P and dP count -lambda times
        if constexpr (kDiff) mul = -lambda_of<D / 2, kBF16>(terms, lane_id % terms.H);
        [[maybe_unused]] int known = 0, last_start = 0;  // distances in the table; of the open bucket
        [[maybe_unused]] float last_bias = 0.f;
        if constexpr (kBias) {
            table.template load<kBF16>(terms, lane_id % terms.H, tid, kElt);
            named_barrier(2, kElt);
            known = table.spread(terms.n, S, tid, kElt);
            named_barrier(2, kElt);
            last_start = table.start[terms.n - 1];
            last_bias = table.bias[terms.n - 1];
        }
        [[maybe_unused]] float *win = reinterpret_cast<float *>(smem + L::kOffWin) + warp * kWindow;
        [[maybe_unused]] const int wlane = tid & 31;
        int u = 0;
        for (; ok; ++u) {
            // (all lanes together: one whose wait ran out must not leave the others to a warp-wide step)
            const bool there = mbar_wait(BAR_S_FULL(u & 1), (u >> 1) & 1, flags);
            if (!__all_sync(0xffffffffu, there)) { ok = false; break; }
            const int i = meta_j[u % kMetaRing];
            const int fl = meta_f[u % kMetaRing];
            if (i < 0) break;
            const int s = u % L::kRing;
            // the step's log-sum-exp and Delta rows arrived with its Q and dO blocks
            const bool rows_there = mbar_wait(BAR_FULL(s), (u / L::kRing) & 1, flags);
            if (!__all_sync(0xffffffffu, rows_there)) { ok = false; break; }
            tc_fence_after();
            const bool in_col = row_exists && ((fl >> half) & 1);  // warp-uniform
            const uint32_t s_at = tmem + t_lane + (kDiff ? diff_slot(u, 0) : s_col(u & 1)) + col0;
            const uint32_t dp_at = tmem + t_lane + (kDiff ? diff_slot(u, 2) : dp_col(u & 1)) + col0;
            uint32_t pw[16], dw[16];
            [[maybe_unused]] uint32_t dw2[16];
            __syncwarp();
            if (in_col) {
                const float *ls = lse_s + s * (L::kRowBytes / 4) + col0;
                const float *dl = delta_s + s * (L::kRowBytes / 4) + col0;
                // the bias: one constant for the step, or a window (query c at distance d_lo + 31 + c - wlane)
                [[maybe_unused]] bool near = false;
                [[maybe_unused]] float off = 0.f;
                [[maybe_unused]] const float *wp = nullptr;
                if constexpr (kBias) {
                    const int d_lo = (i - key_block) * kBlock - (warp & 1) * 32 - 31;
                    // (the diagonal block goes with the near steps, which mask)
                    near = i == key_block || last_start > d_lo;
                    if (near) wp = window_at(win, table, known, terms.n, d_lo, wlane) + 31 - wlane + col0;
                    else off = last_bias;
                }
                const float bias_at = off, times = mul;
                const int hidden = i == key_block ? k_in - col0 : 0;  // queries before this one do not see the key
                auto step = [&, bias_at, times, wp, ls, dl, hidden](auto is_near, auto is_diagonal) {
                    constexpr bool kNear = decltype(is_near)::value, kDiagonal = decltype(is_diagonal)::value;
                    uint32_t sr[32], pr[32];
                    if constexpr (kDiff) {
                        uint32_t sr2[32];
                        tmem_ld32_three(s_at, sr, tmem + t_lane + diff_slot(u, 1) + col0, sr2, dp_at, pr);
                        tc_fence_before();
                        mbar_arrive(BAR_LOADED(u & 1));
#pragma unroll
                        for (int t = 0; t < 16; ++t) {
                            float p[2], ds1[2], ds2[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int c = 2 * t + e;  // query token within block i, from col0
                                const float dp = __uint_as_float(pr[c]);
                                float p1 = ex2_approx(fmaf(__uint_as_float(sr[c]), scale_log2, -ls[c]));
                                float p2 = ex2_approx(fmaf(__uint_as_float(sr2[c]), scale_log2, -ls[64 + c]));
                                if constexpr (kDiagonal) {
                                    p1 = c < hidden ? 0.f : p1;
                                    p2 = c < hidden ? 0.f : p2;
                                }
                                p2 *= times;
                                p[e] = p1 + p2;
                                ds1[e] = p1 * (dp - dl[c]);
                                ds2[e] = p2 * (dp - dl[64 + c]);
                            }
                            pw[t] = pack16x2<kBF16>(p[0], p[1]);
                            dw[t] = pack16x2<kBF16>(ds1[0], ds1[1]);
                            dw2[t] = pack16x2<kBF16>(ds2[0], ds2[1]);
                        }
                    } else {
                        tmem_ld32_pair(s_at, sr, dp_at, pr);
#pragma unroll
                        for (int t = 0; t < 16; ++t) {
                            float p[2], ds[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int c = 2 * t + e;  // query token within block i, from col0
                                const float l2 = ls[c];
                                const float x = __uint_as_float(sr[2 * t + e]), dp = __uint_as_float(pr[2 * t + e]);
                                float z;
                                if constexpr (kNear) z = fmaf(x, scale_log2, wp[c]) - l2;
                                else if constexpr (kBias) z = fmaf(x, scale_log2, bias_at - l2);
                                else z = fmaf(x, scale_log2, -l2);
                                p[e] = ex2_approx(z);
                                if constexpr (kDiagonal) p[e] = c < hidden ? 0.f : p[e];
                                ds[e] = p[e] * (dp - dl[c]);
                            }
                            pw[t] = pack16x2<kBF16>(p[0], p[1]);
                            dw[t] = pack16x2<kBF16>(ds[0], ds[1]);
                        }
                    }
                };
                if constexpr (kBias) {
                    if (near) step(std::true_type{}, std::true_type{});
                    else step(std::false_type{}, std::false_type{});
                } else {
                    if (i == key_block) step(std::false_type{}, std::true_type{});
                    else step(std::false_type{}, std::false_type{});
                }
            } else {
#pragma unroll
                for (int t = 0; t < 16; ++t) {
                    pw[t] = dw[t] = 0u;
                    if constexpr (kDiff) dw2[t] = 0u;
                }
                if constexpr (kDiff) mbar_arrive(BAR_LOADED(u & 1));
            }
            __syncwarp();
            tmem_st16(dp_at, dw);  // dS^T over the first 16 of this warp's columns of dP^T
            if constexpr (kDiff) {
                tmem_st16(dp_at + 16, dw2);  // dS2^T over its other 16
                const uint32_t to = sP + (u & 1) * L::kPBytes + row * 128;  // P^T as a left operand, SW128
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    st_shared_v4(to + ((((uint32_t)(col0 >> 3) + q) ^ (uint32_t)(row & 7)) << 4), pw[4 * q], pw[4 * q + 1],
                                 pw[4 * q + 2], pw[4 * q + 3]);
                fence_proxy_async_smem();
            } else {
                tmem_st16(s_at, pw);  // P^T over the first 16 of those of S^T
            }
            tc_fence_before();
            mbar_arrive(BAR_P_FULL(u & 1));
        }
        if (!ok) *abort_flag = 1;
        bool acc_valid = false;
        if (ok && u > 0) {
            // the last two steps' accumulations: those before had completed when the last step's
            // products did
            acc_valid = mbar_wait(BAR_DONE((u - 1) & 1), ((u - 1) >> 1) & 1, flags) &&
                        (u < 2 || mbar_wait(BAR_DONE(u & 1), ((u - 2) >> 1) & 1, flags));
            if (!acc_valid) *abort_flag = 1;
        }
        // one decision for all elementwise warps (the section below has a barrier of its own)
        if (!named_barrier_or(1, kElt, *abort_flag != 0)) {
            tc_fence_after();
            __syncwarp();
            // every product that read K and V has completed: their tiles stage dK and dV
            stage_rows<D, kBF16>(tmem + t_lane, kDVCol, acc_valid, 1.f, sV, row, tid >> 7);
            stage_rows<D, kBF16>(tmem + t_lane, kDKCol, acc_valid, scale, sK, row, tid >> 7);
            fence_proxy_async_smem();
            named_barrier(1, kElt);
            if (tid == 0) {
#pragma unroll
                for (int c = 0; c < L::kChunks; ++c) {
                    tma_store_3d(&tmdV, c * 64, ka * kBlock, lane_id, sV + c * 16384);
                    tma_store_3d(&tmdK, c * 64, ka * kBlock, lane_id, sK + c * 16384);
                    if (has_b) {
                        tma_store_3d(&tmdV, c * 64, kb * kBlock, lane_id, sV + c * 16384 + 8192);
                        tma_store_3d(&tmdK, c * 64, kb * kBlock, lane_id, sK + c * 16384 + 8192);
                    }
                }
                tma_store_commit();
                tma_store_wait_read();
            }
        }
    }
#undef BAR_FULL
#undef BAR_EMPTY
#undef BAR_S_FULL
#undef BAR_P_FULL
#undef BAR_DONE
#undef BAR_LOADED
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) {
        raise_status(flags, kDevTimeout);
        atomicExch(flags.abort_epoch, flags.epoch);
    }
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}


template <int D, bool kBF16, class Terms>
tsa_status launch_grad_kernels(const BwdLaunch &a, const Terms &terms) {
    auto kq = bwd_dq_kernel<D, kBF16, Terms>;
    auto kkv = bwd_dkv_kernel<D, kBF16, Terms>;
    constexpr int kDqBytes = DqSmem<D, Terms>::kBytes, kDkvBytes = DkvSmem<D, Terms>::kBytes;
    static std::atomic<unsigned long long> q_ready{0}, kv_ready{0};
    if (!allow_smem(q_ready, reinterpret_cast<const void *>(kq), kDqBytes) ||
        !allow_smem(kv_ready, reinterpret_cast<const void *>(kkv), kDkvBytes))
        return TSA_ERR_CUDA;
    const unsigned tiles = (unsigned)((a.nb + 1) / 2);
    const dim3 grid((unsigned)a.lanes, tiles);
    const float scale_log2 = a.scale * kLog2e;
    kq<<<grid, kThreads, kDqBytes, a.stream>>>(*a.tmQ128, *a.tmdO128, *a.tmK64, *a.tmV64, *a.tmdQ64, a.row_ptr,
                                               a.col_idx, a.vlen, a.lse_pad, a.delta, a.nb, a.scale, scale_log2,
                                               a.partial, a.flags, terms);
    kkv<<<grid, kThreads, kDkvBytes, a.stream>>>(*a.tmK64, *a.tmV64, *a.tmQ64, *a.tmdO64, *a.tmdK64, *a.tmdV64,
                                                 a.col_ptr, a.row_idx, a.pairs, a.lse_pad, a.delta, a.nb, a.S, a.scale,
                                                 scale_log2, a.flags, terms);
    return cudaGetLastError() == cudaSuccess ? TSA_OK : TSA_ERR_CUDA;
}

template <class Terms>
tsa_status launch_gradients(const BwdLaunch &a, const Terms &terms) {
    if (a.D == 64) return a.bf16 ? launch_grad_kernels<64, true>(a, terms) : launch_grad_kernels<64, false>(a, terms);
    if (a.D == 128)
        return a.bf16 ? launch_grad_kernels<128, true>(a, terms) : launch_grad_kernels<128, false>(a, terms);
    return TSA_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace tsa
