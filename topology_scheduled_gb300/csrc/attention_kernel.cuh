// attention_kernel.cuh -- scheduled causal attention forward on tcgen05 tensor cores (sm_103a).
//
// Method ("Add topology-derived sparse attention kernel" (triton-lang/kernels#22), Summary,
// and the port note on the PR's mirror page): for every 64-token query block visit only the
// key blocks of its CSR row, keep a running row maximum and denominator, rescale by
// exp(m_prev - m_new), and mask keys after the query token inside the diagonal block.
//
// GB300 design (not the pages' Triton kernel):
//  * Tile.  One CTA computes 128 query rows: query blocks 2p and 2p+1 of one lane, because
//    tcgen05 runs at full rate at M = 128.  It walks the sorted union of the two CSR rows; a
//    key block in only one row is masked for the other half (each half is two whole warps).
//  * Warp roles (192 threads).  Warp 4 produces: one thread TMA-loads Q once and the K and V
//    tiles of each visited block into two-stage rings of their own (128-byte swizzle), polling
//    both rings so that neither stream waits behind the other.  Warp 5 issues the MMAs from
//    one thread: S = Q K^T (M128 N64 K=D, both operands in shared memory) into one of two TMEM
//    S buffers, and O += P V (M128 N=D K64) with P read from TMEM.  Warps 0-3 run the online
//    softmax, one row per thread: tcgen05.ld of the S row, exp2 with the scale folded in, the
//    new P written back over the S buffer in the input dtype with tcgen05.st.
//  * Pipeline.  The MMA warp issues QK(u+1) before PV(u), so the tensor core computes the next
//    scores while the softmax warps work on the current ones.  K and V have rings of their
//    own: a K stage is refilled as soon as its QK is done, so the next key tile is already
//    resident when the MMA warp reaches it.  Hand-offs are mbarriers: k_full/k_empty and
//    v_full/v_empty (producer <-> MMA), s_full (MMA -> softmax, also carries the end of the
//    row union), p_full (softmax -> MMA), o_done (PV completion, for rescaling and the
//    epilogue).
//  * Lazy rescale.  O and the denominator are rescaled only when a row's maximum grows by more
//    than 2^30 (bf16) or 2^15 (f16); the final O / l uses the same stale maximum, so the result
//    is unchanged.  The decision is per row but TMEM loads/stores are warp-collective, so a
//    warp rescales when any of its rows must (factor 1 for the others).
//  * Precision.  Scores, maxima, denominators and O are binary32.  P is rounded to the input dtype for its
//    product with V: tcgen05 multiplies 16-bit operands at twice the rate of the 32-bit ones, which keep 10
//    bits.  An output is off by at most that rounding of the weights and its own.
//  * Epilogue.  O / l rounded to the input dtype, staged in the Q tile, TMA-stored per block;
//    optionally the row's log-sum-exp (m + log l), which the backward pass recomputes P from.
//  * Partial last block (S not a multiple of 64).  The maps see [lanes, S, D] as three dimensions: rows
//    past a lane's end read as zero, whatever the next lane holds, and are not written.  As keys
//    they never weigh, since the block is visited only as the diagonal block of the last row, where
//    the causal mask already drops keys after the query token.
//  * Two CTAs share an SM, so one CTA's softmax also overlaps the other's MMAs.
//
// The same kernel carries the score terms of score_terms.cuh:
//  * Bias by buckets of the distance q - k.  Far enough from the diagonal all keys of a step lie in the
//    open last bucket for all rows of a warp, and then the bias is one constant, folded into the FMA
//    that subtracts the row maximum: such a step costs what a plain one does.  Otherwise every thread
//    reads its 64 biases from a table by distance in shared memory, lane by lane consecutive addresses
//    (no bank conflicts), one FMA per score.  The softmax warps fill the table (the first 2048 distances
//    at most) while the first tiles are on their way; beyond it a warp lays out the 95 distances of its
//    step.
//  * Differential attention.  A CTA takes one query block and both maps: rows 0-63 of the tile are
//    the block's first map, rows 64-127 its second.  With Q laid out block-diagonally
//    ([q1 0; 0 q2], zeros written by the softmax warps) the product with the unsplit K rows gives
//    q1.k1 above and q2.k2 below, and P V gives both maps' outputs from one V tile, so a step costs
//    what a plain one of the same D does and no row union is needed.  The zeros double the score
//    product's multiplications, but a 64-row product would run at half the rate: the tensor time
//    is the same.  The epilogue subtracts the lower rows from the upper through shared memory.
//    At D = 64, many tiles and short rows three CTAs share an SM (kThree), as two leave half of the issue slots empty.
//    Three leave 96 registers per thread and 128 TMEM columns per CTA (one allocation, so that no CTA
//    waits for columns while it holds some).  So a softmax thread takes its 64 scores in two parts of
//    32, the first one read twice (for the maximum and for the weights); there is one S buffer beside
//    O, the next scores are computed once the softmax warps have read S, and P goes through 16 KB of
//    shared memory, written once the product that read the last one is done (figures at launch_gran).  P
//    over the one S buffer, which makes every step run in series, lost to two CTAs, and a bias gains
//    nothing, as the steps near the diagonal then add it twice.
// Measured at [1, 32, 32768, 128] bf16, 14.5 blocks a row: plain 0.42 ms (1190 TFLOP/s on visited blocks),
// biased 0.44 ms, differential 0.85 ms, 0.90 ms with what its backward needs (twice the tiles: 1100
// TFLOP/s executed).  Bound by the softmax warps' chain of a step beside a tensor pipe that is active for
// 44 to 53 % of the time: the 64-column score product runs at 2/3 of the full rate.
// Every mbarrier wait is bounded; on a timeout the CTA records TSA_ERR_TIMEOUT, drains its
// in-flight copies and MMAs (bounded), frees TMEM and returns.
#pragma once

#include <cfloat>
#include <climits>
#include <type_traits>

#include "score_terms.cuh"
#include "tsa_device.cuh"
#include "tsa_internal.h"

namespace tsa {
namespace {

constexpr int kRows = 128;            // query rows per CTA (two 64-token query blocks)
constexpr int kBlock = 64;            // tokens per key / query block
constexpr int kKStages = 2;           // K ring depth
constexpr int kVStages = 2;           // V ring depth
constexpr int kThreads = 192;         // 4 softmax warps + producer warp + MMA warp
constexpr int kProducerWarp = 4;
constexpr int kMmaWarp = 5;
// Lazy-rescale threshold (log2 units): O and the denominator are rescaled only when a row's
// maximum grows past the one they are scaled to by more than this, so p stays at most 2^30
// (bf16: far inside its range and the fp32 accumulators') or 2^15 (f16: below its largest
// finite value, 65504).  Rescales cost a wait for the running PV product and a pass over O in
// TMEM; keys drawn around distinct cluster means made a small threshold (2^8) rescale often.
template <bool kBF16>
__device__ __forceinline__ constexpr float rescale_log2() { return kBF16 ? 30.0f : 15.0f; }

// kThree: the layout for three CTAs per SM (differential, D = 64)
template <int D, bool kThree>
struct AttnSmem {
    static constexpr int kD = D;
    static constexpr int kChunks = D / 64;            // 64-element (128 B) column chunks
    static constexpr int kQBytes = kRows * D * 2;     // Q tile, later the O staging tile
    static constexpr int kKVBytes = kBlock * D * 2;   // one K or V tile
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + kQBytes;                // kKStages tiles
    static constexpr int kOffV = kOffK + kKStages * kKVBytes;    // kVStages tiles
    static constexpr int kOffP = kOffV + kVStages * kKVBytes;    // kOneS: a step's P
    static constexpr int kOffMeta = kOffP + (kThree ? kRows * kBlock * 2 : 0);
    static constexpr int kMetaBytes = 256;
    static constexpr int kOffTable = kOffMeta + kMetaBytes;           // BucketTable (bias only)
    static constexpr int kOffWin = kOffTable + kBucketTableBytes;     // 4 windows (bias only)
    static constexpr int kEnd = kThree ? kOffTable : kOffWin + 4 * kWindow * 4;
    // With the 1 KB that each CTA reserves, 228 KB hold two (D = 128) or three of these; at least 512
    // bytes are left for aligning the dynamic shared-memory base to 1024 (the kernel checks the actual
    // alignment and reports kDevSmemAlign if it does not fit).
    static constexpr int kBytes = D == 128 ? 115712 : 66688;
    static_assert(kEnd + 512 <= kBytes, "smem");
    // the K ring holds the second map's fp32 output rows in the differential epilogue
    static_assert(kKStages * kKVBytes >= kBlock * D * 4, "exchange");
    static constexpr bool kOneS = kThree;
    static constexpr int kCtas = kOneS ? 3 : 2;  // per SM
    // S0 | S1 | O, P_b over the first 32 columns of S_b; or S | O, and P in shared memory
    static constexpr int kTmemCols = kOneS ? 128 : 256;
    static constexpr int kOCol = kOneS ? 64 : 128;

    static constexpr int kPart = kOneS ? 32 : 64;  // keys of a step that a softmax thread holds at a time

    __device__ static __forceinline__ uint32_t s_col(int b) { return !kOneS && b ? 64u : 0u; }
};

// Meta area layout (byte offsets from kOffMeta).
// Union entries in flight: the producer writes entry v once QK(v - kKStages) is done, while the
// softmax warps may still be about to read entry v - kKStages - 1, so the ring holds more.
constexpr int kMetaRing = 8;
static_assert(kMetaRing >= kKStages + 2, "meta ring shorter than the K ring's lead");
constexpr int kBarQ = 0;
constexpr int kBarKFull = 8;                          // kKStages x 8
constexpr int kBarKEmpty = kBarKFull + 8 * kKStages;  // kKStages x 8
constexpr int kBarVFull = kBarKEmpty + 8 * kKStages;  // kVStages x 8
constexpr int kBarVEmpty = kBarVFull + 8 * kVStages;  // kVStages x 8
constexpr int kBarSFull = kBarVEmpty + 8 * kVStages;  // 2 x 8
constexpr int kBarPFull = kBarSFull + 16;             // 2 x 8
constexpr int kBarODone = kBarPFull + 16;
constexpr int kBarFin = kBarODone + 16;               // (o_done: 2 x 8)
constexpr int kBarQDiag = kBarFin + 8;  // Q is block-diagonal (differential attention)
constexpr int kBarSRead = kBarQDiag + 8;  // the softmax warps have read S (one buffer)
constexpr int kTmemSlot = kBarSRead + 8;
constexpr int kAbortFlag = kTmemSlot + 4;
constexpr int kMetaJ = kAbortFlag + 4;                // kMetaRing x 4
constexpr int kMetaF = kMetaJ + 4 * kMetaRing;        // kMetaRing x 4
static_assert(kMetaF + 4 * kMetaRing <= 256, "meta area");

// Walks the union of two sorted CSR rows (query blocks qa and qa+1), checking the row
// contract on the way.  Used by the producer thread.
//
// With 128-token blocks (coarse) the CTA's two 64-token query blocks are one CSR row p = qa/2,
// and each 128-token key block j of it is visited as the 64-token blocks 2j and 2j+1: both
// for both halves when j < p; on the diagonal (j == p) block 2p for both halves (the token
// mask then holds keys to k <= q in the first half, the second half sees all of it) and block
// 2p+1 for the second half only.  The allowed key set of every token is the 128-block one.
struct RowUnion {
    const int32_t *col;
    int ia, ia_end, ib, ib_end;
    int last_a, last_b, qa, qb;
    bool bad;
    bool coarse, has_b;
    int nb64, pend, pend_flags;

    // kChecked: a row must also lie within the cap entries of col_idx
    template <bool kChecked>
    __device__ void init(const int32_t *row_ptr, const int32_t *col_idx, int qa_, bool has_b_,
                         bool coarse_, int nb64_, int cap) {
        col = col_idx;
        qa = qa_;
        qb = qa_ + 1;
        bad = false;
        coarse = coarse_;
        has_b = has_b_;
        nb64 = nb64_;
        pend = -1;
        pend_flags = 0;
        if (coarse) {
            const int p = qa >> 1;
            ia = row_ptr[p];
            ia_end = row_ptr[p + 1];
            if (ia_end - ia < 0 || ia_end - ia > p + 1 || (kChecked && (ia < 0 || ia_end > cap))) {
                bad = true;
                ia_end = ia;
            }
            ib = ib_end = 0;
            last_a = last_b = -1;
            return;
        }
        ia = row_ptr[qa];
        ia_end = row_ptr[qa + 1];
        if (ia_end - ia < 0 || ia_end - ia > qa + 1 || (kChecked && (ia < 0 || ia_end > cap))) {
            bad = true;
            ia_end = ia;
        }
        if (has_b) {
            ib = row_ptr[qb];
            ib_end = row_ptr[qb + 1];
            if (ib_end - ib < 0 || ib_end - ib > qb + 1 || (kChecked && (ib < 0 || ib_end > cap))) {
                bad = true;
                ib_end = ib;
            }
        } else {
            ib = ib_end = 0;
        }
        last_a = last_b = -1;
    }

    // Next key block of the union and its membership bits (1: row qa, 2: row qb); -1 at end.
    __device__ int next(int &flags) {
        int ja = INT_MAX, jb = INT_MAX;
        if (ia < ia_end) {
            ja = __ldg(col + ia);
            if (ja <= last_a || ja > qa) { bad = true; ia_end = ia; ja = INT_MAX; }
        }
        if (ib < ib_end) {
            jb = __ldg(col + ib);
            if (jb <= last_b || jb > qb) { bad = true; ib_end = ib; jb = INT_MAX; }
        }
        if (ja == INT_MAX && jb == INT_MAX) { flags = 0; return -1; }
        const int j = ja < jb ? ja : jb;
        flags = (ja == j ? 1 : 0) | (jb == j ? 2 : 0);
        if (ja == j) { last_a = ja; ++ia; }
        if (jb == j) { last_b = jb; ++ib; }
        return j;
    }

    // 64-token entries of a 128-token CSR row (see above).
    __device__ int next_coarse(int &flags) {
        if (pend >= 0) {
            const int j = pend;
            flags = pend_flags;
            pend = -1;
            return j;
        }
        const int p = qa >> 1;
        if (ia >= ia_end) { flags = 0; return -1; }
        const int j = __ldg(col + ia);
        if (j <= last_a || j > p) { bad = true; ia_end = ia; flags = 0; return -1; }
        last_a = j;
        ++ia;
        const int rows = has_b ? 3 : 1;
        flags = rows;
        const int fb = j < p ? rows : (rows & 2);
        if (2 * j + 1 < nb64 && fb != 0) {
            pend = 2 * j + 1;
            pend_flags = fb;
        }
        return 2 * j;
    }

    // The same for query block qa alone: all of block j's 64-token halves that lie at or before it.
    __device__ int next_coarse_single(int &flags) {
        flags = 1;
        if (pend >= 0) {
            const int j = pend;
            pend = -1;
            return j;
        }
        if (ia >= ia_end) { flags = 0; return -1; }
        const int j = __ldg(col + ia);
        if (j <= last_a || j > qa >> 1) { bad = true; ia_end = ia; flags = 0; return -1; }
        last_a = j;
        ++ia;
        if (2 * j + 1 <= qa) pend = 2 * j + 1;
        return 2 * j;
    }
};

// 32-token blocks: the CTA's 128 rows are query blocks r0 .. r0+3 (r0 = 2 qa), and each 64-token
// key block k of the union of their CSR rows carries one bit per (query quarter r, key half h):
// bit 2r + h when row r0 + r holds 32-token key block 2k + h.  Rows are checked as above.
struct RowUnion32 {
    const int32_t *col;
    int pos[4], end[4], last[4];
    int r0;
    bool bad;

    template <bool kChecked>
    __device__ void init(const int32_t *row_ptr, const int32_t *col_idx, int r0_, int nrows, int cap) {
        col = col_idx;
        r0 = r0_;
        bad = false;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            last[r] = -1;
            pos[r] = end[r] = 0;
            if (r < nrows) {
                pos[r] = row_ptr[r0 + r];
                end[r] = row_ptr[r0 + r + 1];
                if (end[r] - pos[r] < 0 || end[r] - pos[r] > r0 + r + 1 ||
                    (kChecked && (pos[r] < 0 || end[r] > cap))) {
                    bad = true;
                    end[r] = pos[r];
                }
            }
        }
    }

    __device__ int head(int r) {
        if (pos[r] >= end[r]) return INT_MAX;
        const int x = __ldg(col + pos[r]);
        if (x <= last[r] || x > r0 + r) { bad = true; end[r] = pos[r]; return INT_MAX; }
        return x;
    }

    __device__ int next(int &flags) {
        int h[4], j = INT_MAX;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            h[r] = head(r);
            j = h[r] < j ? h[r] : j;
        }
        flags = 0;
        if (j == INT_MAX) return -1;
        const int k = j >> 1;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (h[r] == 2 * k + hh) {
                    flags |= 1 << (2 * r + hh);
                    last[r] = h[r];
                    ++pos[r];
                    h[r] = head(r);
                }
            }
        }
        return k;
    }
};

// The producer's walk for the CSR's block size kGran (0: 64, 1: 128, 2: 32 tokens): entries are
// 64-token key blocks with their membership bits -- with 32-token blocks bit 2r + h per (query
// quarter r, key half h), otherwise bit h per 64-row query half h (the whole 64-key step).
// kSingle: the walk of query block qa alone (with 32-token blocks, its two rows).
template <int kGran, bool kSingle>
struct EntryWalk {
    RowUnion u;
    RowUnion32 u32;

    template <bool kChecked>
    __device__ void init(const int32_t *row_ptr, const int32_t *col_idx, int qa, bool has_b, int nb64, int S, int cap) {
        if constexpr (kGran == 2) {
            const int nb32 = (S + 31) / 32;
            const int r0 = 2 * qa;
            constexpr int kMost = kSingle ? 2 : 4;
            u32.template init<kChecked>(row_ptr, col_idx, r0, nb32 - r0 < kMost ? nb32 - r0 : kMost, cap);
        } else {
            u.template init<kChecked>(row_ptr, col_idx, qa, has_b, kGran == 1, nb64, cap);
        }
    }

    __device__ int next(int &flags) {
        if constexpr (kGran == 2) return u32.next(flags);
        else if constexpr (kGran == 1) return kSingle ? u.next_coarse_single(flags) : u.next_coarse(flags);
        else return u.next(flags);
    }

    __device__ bool bad() const {
        if constexpr (kGran == 2) return u32.bad;
        else return u.bad;
    }
};

// Two floats rounded to the 16-bit input dtype, packed (first in the low half); `sum` gets
// the rounded values.
template <bool kBF16>
__device__ __forceinline__ uint32_t pack2(float a, float b, float &sum) {
    if constexpr (kBF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        sum += __low2float(h) + __high2float(h);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        sum += __low2float(h) + __high2float(h);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

template <int D, bool kThree, bool kBF16, int kGran, class Terms>
__global__ void __launch_bounds__(kThreads, AttnSmem<D, kThree>::kCtas)
scheduled_attention_kernel(const __grid_constant__ CUtensorMap tmQ,
                           const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV,
                           const __grid_constant__ CUtensorMap tmO,
                           const __grid_constant__ CUtensorMap tmO2,
                           const int32_t *__restrict__ row_ptr, const int32_t *__restrict__ col_idx, int nnz_cap,
                           bool with_o2, float *__restrict__ lse_out, int nb, int S,
                           float scale_log2, DeviceFlags flags, const __grid_constant__ Terms terms) {
    constexpr bool kBias = Terms::kBias, kDiff = Terms::kDiff;
    constexpr bool kFine = kGran == 2;  // 32-token blocks: masks per (query quarter, key half)
    using L = AttnSmem<D, kThree>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];

    const uint32_t raw_base = smem_u32(smem_raw);
    const uint32_t base = (raw_base + 1023u) & ~1023u;
    constexpr uint32_t kUsed = kBias ? L::kEnd : L::kOffMeta + L::kMetaBytes;
    if (base - raw_base + kUsed > (uint32_t)L::kBytes) {
        if (threadIdx.x == 0) raise_status(flags, kDevSmemAlign);
        return;
    }
    uint8_t *smem = smem_raw + (base - raw_base);
    const uint32_t sQ = base + L::kOffQ;
    const uint32_t sK0 = base + L::kOffK;
    const uint32_t sV0 = base + L::kOffV;
    const uint32_t meta = base + L::kOffMeta;
    volatile int *meta_j = reinterpret_cast<volatile int *>(smem + L::kOffMeta + kMetaJ);
    volatile int *meta_f = reinterpret_cast<volatile int *>(smem + L::kOffMeta + kMetaF);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::kOffMeta + kAbortFlag);
    [[maybe_unused]] const uint32_t bar_q_diag = meta + kBarQDiag;
    [[maybe_unused]] const BucketTable table(smem + L::kOffTable);
    [[maybe_unused]] const uint32_t bar_s_read = meta + kBarSRead;
    const uint32_t bar_q = meta + kBarQ, bar_fin = meta + kBarFin;
#define BAR_K_FULL(s) (meta + kBarKFull + 8u * (uint32_t)(s))
#define BAR_K_EMPTY(s) (meta + kBarKEmpty + 8u * (uint32_t)(s))
#define BAR_V_FULL(s) (meta + kBarVFull + 8u * (uint32_t)(s))
#define BAR_V_EMPTY(s) (meta + kBarVEmpty + 8u * (uint32_t)(s))
#define BAR_S_FULL(b) (meta + kBarSFull + 8u * (uint32_t)(b))
#define BAR_P_FULL(b) (meta + kBarPFull + 8u * (uint32_t)(b))
#define BAR_O_DONE(b) (meta + kBarODone + 8u * (uint32_t)(b))

    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const int lane_id = blockIdx.y;                  // attention lane (batch * head)
    const int last_tile = (int)gridDim.x - 1;        // a tile: two query blocks (kDiff: one, both maps)
    const int qa = (last_tile - (int)blockIdx.x) * (kDiff ? 1 : 2);  // longest rows first
    const bool has_b = !kDiff && qa + 1 < nb;

    // The first global reads are issued together and waited for at the barrier below: whether
    // the launch already gave up elsewhere (one thread reads the flag, so the whole CTA takes
    // the same branch), and the producer's CSR rows.
    const bool gave_up = tid == 0 && *reinterpret_cast<volatile unsigned *>(flags.abort_epoch) == flags.epoch;
    EntryWalk<kGran, kDiff> ruk, ruv;  // the producer's walks of the row union, one per stream
    if (warp == kProducerWarp && elect_one()) {
        ruk.template init<kBias || kDiff>(row_ptr, col_idx, qa, has_b, nb, S, nnz_cap);
        ruv.template init<kBias || kDiff>(row_ptr, col_idx, qa, has_b, nb, S, nnz_cap);
    }

    if (tid == 0) {
        mbar_init(bar_q, 1);
        for (int s = 0; s < kKStages; ++s) {
            mbar_init(BAR_K_FULL(s), 1);
            mbar_init(BAR_K_EMPTY(s), 1);
        }
        for (int s = 0; s < kVStages; ++s) {
            mbar_init(BAR_V_FULL(s), 1);
            mbar_init(BAR_V_EMPTY(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(BAR_S_FULL(b), 1);
            mbar_init(BAR_P_FULL(b), kRows);
            mbar_init(BAR_O_DONE(b), 1);
        }
        mbar_init(bar_fin, 1);
        if constexpr (kDiff) mbar_init(bar_q_diag, kRows);
        if constexpr (L::kOneS) mbar_init(bar_s_read, kRows);
        *abort_flag = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(meta + kTmemSlot, L::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    const bool leave = __syncthreads_or(gave_up);
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::kOffMeta + kTmemSlot);
    if (leave) {  // nothing was issued yet: give the columns back and go
        if (tid == 0) raise_status(flags, kDevTimeout);  // a replayed launch that gave up once says so again
        if (warp == kMmaWarp) tmem_dealloc(tmem, L::kTmemCols);
        return;
    }

    if (warp == kProducerWarp) {
        // ------------------------------------------------------------ producer (TMA)
        // One thread, two independent streams: the K tile of union entry v goes into K stage
        // v % kKStages as soon as QK(v - kKStages) has freed it, the V tile into V stage
        // v % kVStages as soon as PV(v - kVStages) has; the thread polls both rings, so a K
        // load never waits behind a V stage.
        if (elect_one()) {
            tma_prefetch_desc(&tmQ);
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
            tma_prefetch_desc(&tmO);
            mbar_arrive_expect_tx(bar_q, L::kQBytes);
#pragma unroll
            for (int c = 0; c < L::kChunks; ++c) {
                tma_load_3d(sQ + c * 16384, &tmQ, c * 64, qa * kBlock, lane_id, bar_q);
                if constexpr (kDiff)  // 64-row boxes: the block again, for the second map
                    tma_load_3d(sQ + c * 16384 + 8192, &tmQ, c * 64, qa * kBlock, lane_id, bar_q);
            }
            bool ok = true, k_done = false, v_done = false;
            int kv = 0, vv = 0;  // next union entry of each stream
            unsigned long long t_idle = 0;
            for (uint32_t it = 0; !(k_done && v_done); ++it) {
                bool progress = false;
                if (!k_done && (kv < kKStages ||
                                mbar_try_wait(BAR_K_EMPTY(kv % kKStages), (uint32_t)((kv / kKStages) - 1) & 1u))) {
                    const int s = kv % kKStages;
                    int f = 0;
                    const int j = ruk.next(f);
                    meta_j[kv % kMetaRing] = j;
                    meta_f[kv % kMetaRing] = f;
                    if (j < 0) {
                        mbar_arrive(BAR_K_FULL(s));  // the end marker travels with the K ring
                        k_done = true;
                    } else {
                        mbar_arrive_expect_tx(BAR_K_FULL(s), L::kKVBytes);
#pragma unroll
                        for (int c = 0; c < L::kChunks; ++c)
                            tma_load_3d(sK0 + s * L::kKVBytes + c * 8192, &tmK, c * 64, j * kBlock, lane_id,
                                             BAR_K_FULL(s));
                        ++kv;
                    }
                    progress = true;
                }
                if (!v_done && (vv < kVStages ||
                                mbar_try_wait(BAR_V_EMPTY(vv % kVStages), (uint32_t)((vv / kVStages) - 1) & 1u))) {
                    const int s = vv % kVStages;
                    int f = 0;
                    const int j = ruv.next(f);
                    if (j < 0) {
                        v_done = true;
                    } else {
                        mbar_arrive_expect_tx(BAR_V_FULL(s), L::kKVBytes);
#pragma unroll
                        for (int c = 0; c < L::kChunks; ++c)
                            tma_load_3d(sV0 + s * L::kKVBytes + c * 8192, &tmV, c * 64, j * kBlock, lane_id,
                                             BAR_V_FULL(s));
                        ++vv;
                    }
                    progress = true;
                }
                // bounded: give up after kWaitTimeoutNs without progress, or when the launch did
                if (progress) {
                    t_idle = 0;
                } else if ((it & 63u) == 0u) {
                    const unsigned long long now = globaltimer();
                    if (t_idle == 0) t_idle = now;
                    if (now - t_idle > kWaitTimeoutNs ||
                        *reinterpret_cast<volatile unsigned *>(flags.abort_epoch) == flags.epoch) {
                        ok = false;
                        break;
                    }
                }
            }
            if (ruk.bad()) raise_status(flags, kDevBadSchedule);
            if (!ok) {
                // Drain: wait (bounded) for every load issued into the rings.
                *abort_flag = 1;
                (void)mbar_wait_timed(bar_q, 0);
                for (int w = kv - kKStages; w < kv; ++w)
                    if (w >= 0) (void)mbar_wait_timed(BAR_K_FULL(w % kKStages), (w / kKStages) & 1);
                for (int w = vv - kVStages; w < vv; ++w)
                    if (w >= 0) (void)mbar_wait_timed(BAR_V_FULL(w % kVStages), (w / kVStages) & 1);
            }
        }
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMA issuer
        if (elect_one()) {
            constexpr uint32_t kIdescQK = idesc_f16(kBF16, 128, 64, false);
            constexpr uint32_t kIdescPV = idesc_f16(kBF16, 128, D, true);
            const uint64_t q_desc = sdesc_sw128(sQ, 16, 1024), k_desc = sdesc_sw128(sK0, 16, 1024),
                           v_desc = sdesc_sw128(sV0, 8192, 1024);
            [[maybe_unused]] const uint64_t p_desc = sdesc_sw128(base + L::kOffP, 16, 1024);
            bool ok = mbar_wait(bar_q, 0, flags);
            if constexpr (kDiff) ok = ok && mbar_wait(bar_q_diag, 0, flags);
            int u = 0;
            bool have = false;  // entry u exists and QK(u) was issued
            // QK(u): S_{u%2} = Q K_u^T; frees K stage u % kKStages when done
#define ISSUE_QK(uu)                                                                              \
    do {                                                                                          \
        const int s_ = (uu) % kKStages;                                                           \
        tc_fence_after();                                                                         \
        _Pragma("unroll") for (int kk = 0; kk < D / 16; ++kk) {                                   \
            const uint64_t a_ = sdesc_at(q_desc, (kk >> 2) * 16384 + (kk & 3) * 32);              \
            const uint64_t b_ = sdesc_at(k_desc, s_ * L::kKVBytes + (kk >> 2) * 8192 + (kk & 3) * 32); \
            tc_mma_ss(tmem + L::s_col((uu) & 1), a_, b_, kIdescQK, kk > 0 ? 1u : 0u);               \
        }                                                                                         \
        tc_commit(BAR_S_FULL((uu) & 1));                                                          \
        tc_commit(BAR_K_EMPTY(s_));                                                               \
    } while (0)
            // The end of the row union is passed to the softmax warps as an s_full arrival
            // without scores (they read the end marker from the meta ring).
            if (ok) {
                ok = mbar_wait(BAR_K_FULL(0), 0, flags);
                if (ok) {
                    // test hook: the launch's first CTA withholds its first scores (no product,
                    // no arrival), so its softmax warps' bounded wait runs out
                    const bool withhold = flags.inject == 1u && blockIdx.x == 0 && blockIdx.y == 0;
                    if (meta_j[0] >= 0 && !withhold) {
                        ISSUE_QK(0);
                        have = true;
                    } else if (meta_j[0] < 0) {
                        mbar_arrive(BAR_S_FULL(0));
                    }
                }
            }
            while (ok && have) {
                // next scores first, so they overlap the softmax of u
                bool next = false;
                const int s1 = (u + 1) % kKStages;
                ok = mbar_wait(BAR_K_FULL(s1), ((u + 1) / kKStages) & 1, flags);
                if (!ok) break;
                if (meta_j[(u + 1) % kMetaRing] >= 0) {
                    if constexpr (L::kOneS) ok = mbar_wait(bar_s_read, u & 1, flags);
                    if (!ok) break;
                    ISSUE_QK(u + 1);
                    next = true;
                } else {
                    mbar_arrive(BAR_S_FULL((u + 1) & 1));
                }
                // O += P_u V_u once the softmax has written P_u and V_u has landed
                ok = mbar_wait(BAR_P_FULL(u & 1), (u >> 1) & 1, flags);
                if (!ok) break;
                const int s = u % kVStages;
                ok = mbar_wait(BAR_V_FULL(s), (u / kVStages) & 1, flags);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint64_t b = sdesc_at(v_desc, s * L::kKVBytes + kk * 2048);
                    if constexpr (L::kOneS)
                        tc_mma_ss(tmem + L::kOCol, sdesc_at(p_desc, kk * 32), b, kIdescPV, (u > 0 || kk > 0) ? 1u : 0u);
                    else
                        tc_mma_ts(tmem + L::kOCol, tmem + L::s_col(u & 1) + kk * 8, b, kIdescPV,
                                  (u > 0 || kk > 0) ? 1u : 0u);
                }
                tc_commit(BAR_V_EMPTY(s));
                tc_commit(BAR_O_DONE(u & 1));
                have = next;
                ++u;
            }
#undef ISSUE_QK
            if (!ok) *abort_flag = 1;
            // all tensor-core work of this CTA has completed once this arrives
            tc_commit(bar_fin);
            (void)mbar_wait_timed(bar_fin, 0);
        }
    } else {
        // ------------------------------------------------------------ softmax (warps 0-3)
        const int half = tid >> 6;               // 0: block qa, 1: block qa+1 (kDiff: the two maps of qa)
        const int my_block = kDiff ? qa : qa + half;
        const bool row_exists = kDiff || half == 0 || has_b;
        const int member = kDiff ? 0 : half;     // the membership bit of this thread's row
        const int row_in = kDiff ? tid & 63 : tid;  // this thread's token, from the tile's first
        const uint32_t t_lane = (uint32_t)(warp * 32) << 16;  // this warp's TMEM lane quarter
        // maximum the accumulators are scaled to (log2).  Below any finite score, but finite: where all scores so
        // far are -inf their weights are 2^(-inf + FLT_MAX) = 0
        float m_used = -FLT_MAX;
        float l_sum = 0.f;                       // running denominator
        [[maybe_unused]] float l_exact = 0.f;    // the same from the weights before their rounding
        bool ok = true;
        [[maybe_unused]] float lam = 0.f;
        if constexpr (kDiff) {
            // Q's off-diagonal halves become zero once its copy has landed
            lam = lambda_of<D / 2, kBF16>(terms, lane_id % terms.H);
            const bool landed = mbar_wait(bar_q, 0, flags);
            ok = __all_sync(0xffffffffu, landed);
            if (ok) {
                keep_diagonal<D>(sQ, tid);
                fence_proxy_async_smem();
                mbar_arrive(bar_q_diag);
            }
        }
        [[maybe_unused]] int known = 0, last_start = 0;  // distances in the table; of the open bucket
        [[maybe_unused]] float last_bias = 0.f;
        if constexpr (kBias) {
            table.template load<kBF16>(terms, lane_id % terms.H, tid, kRows);
            named_barrier(2, kRows);
            known = table.spread(terms.n, (qa + 2) * kBlock, tid, kRows);
            named_barrier(2, kRows);
            last_start = table.start[terms.n - 1];
            last_bias = table.bias[terms.n - 1];
        }
        [[maybe_unused]] float *win = reinterpret_cast<float *>(smem + L::kOffWin) + warp * kWindow;
        constexpr int kPart = L::kPart;
        constexpr bool kOneS = L::kOneS;
        int u = 0;
        for (; ok; ++u) {
            // (all lanes together: one whose wait ran out must not leave the others to a warp-wide step)
            const bool there = mbar_wait(BAR_S_FULL(u & 1), (u >> 1) & 1, flags);
            if (!__all_sync(0xffffffffu, there)) { ok = false; break; }
            const int j = meta_j[u % kMetaRing];
            const int fl = meta_f[u % kMetaRing];
            if (j < 0) break;
            tc_fence_after();
            // key halves this warp's 32 rows hold (both, with 64- or 128-token blocks)
            const int fq = kFine ? (fl >> (2 * (kDiff ? warp & 1 : warp))) & 3 : ((fl >> member) & 1) * 3;
            const bool in_row = row_exists && fq != 0;  // warp-uniform
            const uint32_t s_addr = tmem + t_lane + L::s_col(u & 1);
            auto store_p = [&](int part, const uint32_t (&pw)[kPart / 2]) {
                if constexpr (kPart == 64) tmem_st32(s_addr, pw);
                else
#pragma unroll
                    for (int q = 0; q < kPart / 8; ++q)  // (rows of 128 bytes, their 16-byte units permuted by row & 7)
                        st_shared_v4(base + L::kOffP + tid * 128 + (((part * 4 + q) ^ (tid & 7)) << 4), pw[4 * q],
                                     pw[4 * q + 1], pw[4 * q + 2], pw[4 * q + 3]);
            };
            // PV(u - 1) has completed: O may be rescaled, and P of one buffer be written
            auto o_done = [&] {
                const bool done = u == 0 || mbar_wait(BAR_O_DONE((u - 1) & 1), ((u - 1) >> 1) & 1, flags);
                return __all_sync(0xffffffffu, done);
            };
            __syncwarp();
            if (in_row) {
                float x[kPart];  // raw scores q.k of a part of the keys
                // scores in log2 units are x * cc + off
                [[maybe_unused]] float cc1 = scale_log2, off = 0.f;
                [[maybe_unused]] const float *wp = nullptr;  // the biases, where they differ
                if constexpr (kBias) {
                    // key c lies at the distance d_lo + 63 + (tid & 31) - c
                    const int d_lo = (qa - j) * kBlock + warp * 32 - 63;
                    if (last_start <= (d_lo > 0 ? d_lo : 0)) {  // all of it in the open last bucket
                        off = last_bias;
                    } else {
                        wp = window_at(win, table, known, terms.n, d_lo, tid & 31) + 63 + (tid & 31);
                        cc1 = 1.f;
                    }
                }
                auto load_scores = [&](int part) {
                    const int c0 = part * kPart;
                    if constexpr (kPart == 64) {
                        uint32_t sr[2][32];
                        tmem_ld32x2(s_addr, sr[0], sr[1]);
#pragma unroll
                        for (int c = 0; c < 64; ++c) x[c] = __uint_as_float(sr[c >> 5][c & 31]);
                    } else {
                        uint32_t sr[32];
                        tmem_ld32(s_addr + c0, sr);
#pragma unroll
                        for (int c = 0; c < 32; ++c) x[c] = __uint_as_float(sr[c]);
                    }
                    if constexpr (kBias) {
                        if (wp != nullptr) {
#pragma unroll
                            for (int c = 0; c < kPart; ++c) x[c] = fmaf(x[c], scale_log2, wp[-c0 - c]);
                        }
                    }
                    if constexpr (kFine) {
                        if (fq != 3) {  // a 32-token key half this row does not hold
#pragma unroll
                            for (int c = 0; c < kPart; ++c)
                                if (!((fq >> ((c0 + c) >> 5)) & 1)) x[c] = -INFINITY;
                        }
                        if (j >= qa) {  // near the diagonal: keys after the query token are masked
                            const int lim = (qa - j) * kBlock + row_in - c0;  // key 64j + c > query 64qa + row_in
#pragma unroll
                            for (int c = 0; c < kPart; ++c)
                                if (c > lim) x[c] = -INFINITY;
                        }
                    } else if (j == my_block) {  // diagonal block: keys after the query token are masked
#pragma unroll
                        for (int c = 0; c < kPart; ++c)
                            if (c > (tid & 63) - c0) x[c] = -INFINITY;
                    }
                };
                float mx = -INFINITY;
#pragma unroll
                for (int part = 0; part < 64 / kPart; ++part) {
                    load_scores(part);
                    float m[(kPart + 2) / 3];
#pragma unroll
                    for (int t = 0; t < kPart / 3; ++t) m[t] = max3f(x[3 * t], x[3 * t + 1], x[3 * t + 2]);
                    if constexpr (kPart == 64) {
                        m[21] = x[63];
                        const float m7a = max3f(max3f(m[0], m[1], m[2]), max3f(m[3], m[4], m[5]),
                                                max3f(m[6], m[7], m[8]));
                        const float m7b = max3f(max3f(m[9], m[10], m[11]), max3f(m[12], m[13], m[14]),
                                                max3f(m[15], m[16], m[17]));
                        mx = max3f(m7a, m7b, max3f(m[18], m[19], fmaxf(m[20], m[21])));
                    } else {
                        m[10] = fmaxf(x[30], x[31]);
                        mx = fmaxf(mx, max3f(max3f(max3f(m[0], m[1], m[2]), max3f(m[3], m[4], m[5]),
                                                   max3f(m[6], m[7], m[8])),
                                             m[9], m[10]));
                    }
                }
                if constexpr (kBias) mx = fmaf(mx, cc1, off);
                else mx *= scale_log2;
                if (kOneS && !o_done()) { ok = false; break; }
                const bool grow = mx > m_used + rescale_log2<kBF16>();
                if (__any_sync(0xffffffffu, grow)) {
                    const float alpha = !grow ? 1.f : ex2_approx(m_used - mx);
                    if (u > 0) {
                        if (!kOneS && !o_done()) { ok = false; break; }
                        tc_fence_after();
                        __syncwarp();
#pragma unroll
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            tmem_ld16(tmem + t_lane + L::kOCol + c, o);
#pragma unroll
                            for (int t = 0; t < 16; ++t) o[t] = __float_as_uint(__uint_as_float(o[t]) * alpha);
                            tmem_st16(tmem + t_lane + L::kOCol + c, o);
                        }
                    }
                    if (grow) {
                        l_sum *= alpha;
                        if constexpr (kDiff) l_exact *= alpha;
                        m_used = mx;
                    }
                }
                // p = 2^(x * scale * log2(e) - m): one packed FMA per pair, exp2 on the MUFU
                const float c1 = kBias ? cc1 : scale_log2;
                float n1 = -m_used;
                if constexpr (kBias) n1 += off;
                const uint64_t cc = f2_pack(c1, c1);
                const uint64_t nm = f2_pack(n1, n1);
                auto weigh = [&, cc, nm](auto exact_too) {
                    constexpr bool kExact = decltype(exact_too)::value;
                    float ls[4] = {0.f, 0.f, 0.f, 0.f};
                    [[maybe_unused]] uint64_t le = f2_pack(0.f, 0.f);
#pragma unroll
                    for (int part = 64 / kPart - 1; part >= 0; --part) {  // the last one is still here
                        if (part < 64 / kPart - 1) load_scores(part);
                        if constexpr (kOneS) {
                            if (part == 0) {
                                tc_fence_before();
                                mbar_arrive(bar_s_read);
                            }
                        }
                        uint32_t pw[kPart / 2];
#pragma unroll
                        for (int t = 0; t < kPart / 2; ++t) {
                            float e0, e1;
                            f2_unpack(f2_fma(f2_pack(x[2 * t], x[2 * t + 1]), cc, nm), e0, e1);
                            const float p0 = ex2_approx(e0), p1 = ex2_approx(e1);
                            if constexpr (kBF16) {
                                const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
                                pw[t] = *reinterpret_cast<const uint32_t *>(&h);
                            } else {
                                const __half2 h = __floats2half2_rn(p0, p1);
                                pw[t] = *reinterpret_cast<const uint32_t *>(&h);
                            }
                            // The denominator sums the rounded P that the PV product uses, so a row
                            // dominated by one key normalizes exactly.
                            add_half<kBF16, false>(ls[(t & 1) * 2], pw[t]);
                            add_half<kBF16, true>(ls[(t & 1) * 2 + 1], pw[t]);
                            if constexpr (kExact) le = f2_add(le, f2_pack(p0, p1));
                        }
                        __syncwarp();
                        store_p(part, pw);
                    }
                    l_sum += (ls[0] + ls[1]) + (ls[2] + ls[3]);
                    if constexpr (kExact) {
                        float e0, e1;
                        f2_unpack(le, e0, e1);
                        l_exact += e0 + e1;
                    }
                };
                // The log-sum-exp of the differential form adds P itself: the backward pass weighs its
                // second map with it to find lambda's gradient, one sum over every row.
                if (kDiff && lse_out) weigh(std::bool_constant<kDiff>{});
                else weigh(std::false_type{});
            } else {
                if constexpr (kOneS) {
                    mbar_arrive(bar_s_read);
                    if (!o_done()) { ok = false; break; }
                }
                const uint32_t pw[kPart / 2] = {};
#pragma unroll
                for (int part = 0; part < 64 / kPart; ++part) store_p(part, pw);
            }
            if constexpr (kOneS) fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(BAR_P_FULL(u & 1));
        }
        if (!ok) *abort_flag = 1;
        // ---- epilogue: O / l in the input dtype, staged in the Q tile, TMA-stored per block
        bool o_valid = false;
        if (ok && u > 0) {
            // the last two PV products (those before had completed when the last scores did)
            o_valid = mbar_wait(BAR_O_DONE((u - 1) & 1), ((u - 1) >> 1) & 1, flags) &&
                      (u < 2 || mbar_wait(BAR_O_DONE(u & 1), ((u - 2) >> 1) & 1, flags));
            if (!o_valid) *abort_flag = 1;
        }
        // one decision for all softmax warps (the section below has a barrier of its own)
        if (!named_barrier_or(1, kRows, *abort_flag != 0)) {
            tc_fence_after();
            const float inv = l_sum > 0.f ? 1.f / l_sum : 0.f;
            const int tok = qa * kBlock + row_in;  // this thread's token (rows of both halves)
            const bool tok_ok = row_exists && tok < S;
            // log-sum-exp of the scaled scores in natural-log units, for the backward pass
            if (lse_out && tok_ok) {
                long long at = (long long)lane_id * S + tok;
                if constexpr (kDiff) at += half * terms.map_rows;
                // (of a row with a NaN score it is NaN, and so are the weights that the backward pass forms)
                lse_out[at] = l_sum == 0.f ? -INFINITY : (m_used + log2f(kDiff ? l_exact : l_sum)) * 0.6931471805599453f;
            }
            const uint32_t sw = (uint32_t)(tid & 7);
            __syncwarp();
            if constexpr (kDiff) {
                // The upper rows' threads finish the first half of the columns, the lower rows' the
                // second: each passes the other's half on in binary32 through the K ring (every
                // product that read it has completed), one 16-byte unit of 64 rows after another.
                // The upper staging rows take O, the lower ones the second map's output.
                constexpr int kW = D / 2;
                const int row = tid & 63;
                float4 *area = reinterpret_cast<float4 *>(smem + L::kOffK) + row;
                auto stage = [&](int col, int to_row, const float (&y)[8]) {
                    float unused = 0.f;
                    st_shared_v4(sQ + (col >> 6) * 16384 + to_row * 128 + ((((col & 63) >> 3) ^ sw) << 4),
                                 pack2<kBF16>(y[0], y[1], unused), pack2<kBF16>(y[2], y[3], unused),
                                 pack2<kBF16>(y[4], y[5], unused), pack2<kBF16>(y[6], y[7], unused));
                };
#pragma unroll
                for (int own = 0; own < 2; ++own) {  // the columns to pass on, then one's own
                    if (own) named_barrier(1, kRows);
                    const int base_col = (half ^ own ^ 1) * kW;
#pragma unroll
                    for (int h = 0; h < kW / 32; ++h) {
                        uint32_t o[32];
                        if (o_valid) {
                            tmem_ld32(tmem + t_lane + L::kOCol + base_col + h * 32, o);
                        } else {
#pragma unroll
                            for (int t = 0; t < 32; ++t) o[t] = 0u;
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            float y[8];
#pragma unroll
                            for (int t = 0; t < 8; ++t) y[t] = __uint_as_float(o[q * 8 + t]) * inv;
                            const int col = base_col + h * 32 + q * 8;
                            if (half && with_o2) stage(col, tid, y);
                            float4 *at = area + (((half ^ own) ? kW / 4 : 0) + h * 8 + q * 2) * 64;
                            if (!own) {
                                at[0] = make_float4(y[0], y[1], y[2], y[3]);
                                at[64] = make_float4(y[4], y[5], y[6], y[7]);
                            } else {
                                const float4 a = at[0], b = at[64];
                                const float z[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                                for (int t = 0; t < 8; ++t) y[t] = half ? fmaf(-lam, y[t], z[t]) : fmaf(-lam, z[t], y[t]);
                                stage(col, row, y);
                            }
                        }
                    }
                }
            } else {
#pragma unroll
            for (int c = 0; c < L::kChunks; ++c) {
                const uint32_t o_row = sQ + c * 16384 + tid * 128;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t o[32];
                    if (o_valid) {
                        tmem_ld32(tmem + t_lane + L::kOCol + c * 64 + h * 32, o);
                    } else {
#pragma unroll
                        for (int t = 0; t < 32; ++t) o[t] = 0u;
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float unused = 0.f;
                        uint32_t w[4];
#pragma unroll
                        for (int t = 0; t < 4; ++t)
                            w[t] = pack2<kBF16>(__uint_as_float(o[q * 8 + 2 * t]) * inv,
                                                __uint_as_float(o[q * 8 + 2 * t + 1]) * inv, unused);
                        const uint32_t chunk16 = (uint32_t)(h * 4 + q);
                        st_shared_v4(o_row + ((chunk16 ^ sw) << 4), w[0], w[1], w[2], w[3]);
                    }
                }
            }
            }
            fence_proxy_async_smem();
            named_barrier(1, kRows);
            if (tid == 0) {
#pragma unroll
                for (int c = 0; c < L::kChunks; ++c) {
                    tma_store_3d(&tmO, c * 64, qa * kBlock, lane_id, sQ + c * 16384);
                    if constexpr (kDiff) {
                        if (with_o2)  // the second map's output, for the backward pass
                            tma_store_3d(&tmO2, c * 64, qa * kBlock, lane_id, sQ + c * 16384 + 8192);
                    } else if (has_b) {
                        tma_store_3d(&tmO, c * 64, (qa + 1) * kBlock, lane_id, sQ + c * 16384 + 8192);
                    }
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
#undef BAR_O_DONE

    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) {
        raise_status(flags, kDevTimeout);
        atomicExch(flags.abort_epoch, flags.epoch);
    }
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kTmemCols);
    }
}

template <int D, bool kThree, bool kBF16, int kGran, class Terms>
tsa_status launch_one(const AttnLaunch &a, const Terms &terms) {
    auto kern = scheduled_attention_kernel<D, kThree, kBF16, kGran, Terms>;
    static std::atomic<unsigned long long> ready{0};
    constexpr int kBytes = AttnSmem<D, kThree>::kBytes;
    if (!allow_smem(ready, reinterpret_cast<const void *>(kern), kBytes)) return TSA_ERR_CUDA;
    const int tiles = Terms::kDiff ? a.nb : (a.nb + 1) / 2;
    dim3 grid((unsigned)tiles, (unsigned)a.lanes);
    kern<<<grid, kThreads, kBytes, a.stream>>>(*a.tmQ, *a.tmK, *a.tmV, *a.tmO, *a.tmO2, a.row_ptr,
                                                            a.col_idx, a.nnz_cap, a.with_o2, a.lse, a.nb, a.S,
                                                            a.scale_log2, a.flags, terms);
    return cudaGetLastError() == cudaSuccess ? TSA_OK : TSA_ERR_CUDA;
}

template <int kGran, class Terms>
tsa_status launch_gran(const AttnLaunch &a, const Terms &terms) {
    if (a.D == 64) {
        if constexpr (Terms::kDiff) {
            // Three CTAs per SM hide more of a tile's start and end, two take less time for a step.  So three for
            // more tiles than run at once, a few times over, and short rows.  us with two / three (f16, rows of
            // random blocks, times without the host's):
            //   blocks a row       2              4              8             16             32             64
            //    512 tiles   11.0 / 11.6    13.8 / 15.4    19.0 / 22.3    28.9 / 30.3    48.9 / 45.4    65.6 / 67.2
            //   1024         19.3 / 17.4    24.6 / 23.2    34.5 / 34.6    51.1 / 51.7    76.6 / 80.5   107.3 / 118.8
            //   2048         33.8 / 29.2    43.4 / 39.6    60.9 / 58.7    92.5 / 92.4   141.6 / 146.1  189.8 / 199.7
            //   8192        134.7 / 109.4  169.3 / 146.8  233.2 / 212.9  349.6 / 335.6  531.0 / 528.8  690.6 / 696.7
            // (64 blocks a head; 16, 32, 128 and 256 differ by a few percent).  The average row is that of the
            // capacity of col_idx, as the host knows no other.
            const int rows = a.gran == 1 ? (a.nb + 1) / 2 : a.gran == 2 ? (a.S + 31) / 32 : a.nb;
            const int block = a.gran == 1 ? 128 : a.gran == 2 ? 32 : 64;
            const bool short_rows = (long long)a.nnz_cap * block <= 16ll * 64 * rows;
            if ((long long)a.nb * a.lanes > 1024 && short_rows)
                return a.bf16 ? launch_one<64, true, true, kGran>(a, terms) : launch_one<64, true, false, kGran>(a, terms);
        }
        return a.bf16 ? launch_one<64, false, true, kGran>(a, terms) : launch_one<64, false, false, kGran>(a, terms);
    }
    if (a.D == 128)
        return a.bf16 ? launch_one<128, false, true, kGran>(a, terms) : launch_one<128, false, false, kGran>(a, terms);
    return TSA_ERR_UNSUPPORTED;
}

template <class Terms>
tsa_status launch_attention(const AttnLaunch &a, const Terms &terms) {
    return a.gran == 2 ? launch_gran<2>(a, terms) : a.gran == 1 ? launch_gran<1>(a, terms) : launch_gran<0>(a, terms);
}

}  // namespace
}  // namespace tsa
