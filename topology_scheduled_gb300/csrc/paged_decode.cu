// paged_decode.cu -- one new token per sequence against a paged key/value cache (include/tsa_cache.h):
// o = softmax(scale q.k) V over the sequence's keys, or those of the blocks its row of a schedule lists.
//
// Bound by memory: 4 D bytes per key and key head.  A key head's queries share them, so the arithmetic,
// 2 D multiply-adds per key and query (4 D in bf16 and 3 D in f16 as issued, a weight's numbers each with a product of their
// own), goes to the tensor cores; one to sixteen multiply-adds a byte are few enough for mma.sync (m16n8k16), whose fragments
// are pieces of rows as they lie in shared memory:
//  * a warp takes 16 keys at a time for up to 8 (or 16) queries.  Scores are S^T = K Q^T, keys as rows.  The
//    order of a contraction is free, so a lane's 16-byte piece of a key serves as two k16 steps' fragment and
//    the same piece of a query as their other operand;
//  * O^T = V^T P^T, dimensions as rows.  V^T's fragment is read transposed (ldmatrix.trans); P^T's is the scores'
//    fragment, transposed (movmatrix);
//  * a weight is a sum of numbers of the inputs' type, each with a product of its own. Three of bf16 are the weight itself,
//    all 24 bits: values that cancel would show the 2^-17 that two lose. Two of f16 are off by 2^-22 of it at most, no more
//    than exp2 is; they are scaled by 2^14 beforehand, so that what is lost is below 2^-39 of the largest weight however
//    small the weight is.  Sums, maxima and denominators are binary32;
//  * a warp copies its keys and values to a ring of its own in shared memory (cp.async), two steps ahead of
//    the one it works on: up to 24 KB in flight per warp, whatever the registers hold.  16 keys of a page are
//    one contiguous 2 D x 16 byte piece; its 16-byte pieces are stored with bits of the row's number
//    exclusive-ored into their place, so that the reads of eight lanes meet all banks once.
// A (sequence, key head, group of queries) is split over the warps of a cluster of thread blocks, whose sums
// are joined through shared memory in a fixed order; where eight blocks a row cannot fill the GPU, several
// clusters share a row, leave their sums in the workspace, and a second kernel joins them.
// Keys at the length and beyond are neither read nor counted.
// Measured (bf16, D = 128): 16 sequences of 8192 keys, 32 heads with keys of their own (2.15 GB) 290-296 us = 7.3 TB/s;
// 64 ragged ones to 8192, 32 heads on 4, 110 us = 6.4; one of 131072, 32 heads on 8, 82-85 us = 6.4. A step is 305
// instructions of a warp (8 queries), 24 % of the issue slots, and the tensor pipe is busy 20 %. (With weights of two
// numbers, and sums left to the tensor cores, 265, 21 and 15 %: 1 to 2 % faster, 14 and 21 % with 16 and 32 queries a key.)
#include <algorithm>
#include <atomic>
#include <climits>

#include "tsa_device.cuh"
#include "tsa_internal.h"

namespace tsa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

constexpr int kStages = 3;                     // of a warp's ring
constexpr int kHalf = 4096;                    // bytes of a step's keys, and of its values
constexpr int kRing = kStages * 2 * kHalf;     // bytes per warp
constexpr int kSmem = kWarps * kRing;

// 16 bytes to shared memory, or 16 zeros.
__device__ __forceinline__ void copy16(uint32_t to, const uint16_t *from, bool there) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_begun() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copies_done() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

__device__ __forceinline__ uint4 load_piece(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}

template <bool kBF16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if constexpr (kBF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of 16-bit elements, two per lane, transposed across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Four 8 x 8 matrices of 16-bit elements, transposed; lane 8 i + r gives the place of matrix i's row r.
__device__ __forceinline__ void load_transposed(uint32_t at, uint32_t (&x)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(at)
                 : "memory");
}

// Two weights as words of the inputs' type whose sum they are: their roundings, and then the roundings of what is left.
template <bool kBF16, int kParts>
__device__ __forceinline__ void in_parts(float a, float b, uint32_t (&w)[kParts]) {
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        if constexpr (kBF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
            a -= __low2float(h);
            b -= __high2float(h);
        } else {
            const __half2 h = __floats2half2_rn(a, b);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
            a -= __low2float(h);
            b -= __high2float(h);
        }
    }
}

template <bool kBF16>
__device__ __forceinline__ void store16(uint16_t *p, float y) {
    if constexpr (kBF16) *p = __bfloat16_as_ushort(__float2bfloat16_rn(y));
    else *p = __half_as_ushort(__float2half_rn(y));
}

// A reference for exponents: the maximum, or 0 where there is no key with weight yet.
__device__ __forceinline__ float reference(float m) { return m == -INFINITY ? 0.f : m; }

// Queries per thread block are 8 kGroups; a warp's step takes 16 kSub keys (4 KB of K either way).
template <int D, bool kBF16, int kGroups>
__global__ void __launch_bounds__(kThreads, 2)
paged_decode_kernel(const __grid_constant__ PagedDecodeLaunch a) {
    constexpr int kSub = D == 64 ? 2 : 1;
    constexpr int kVec = D / 32;   // 16-byte pieces of a key that a lane holds
    constexpr int kTiles = D / 16; // m16 tiles of the output's dimensions
    constexpr int kQ = 8 * kGroups;
    constexpr int kBatch = 32 / kSub;  // a warp's steps whose places it looks up at once
    constexpr int kParts = kBF16 ? 3 : 2;  // numbers that a weight is the sum of
    // A weight is at most 2^(kLift + kSlack) as it is rounded: 2^15 in f16, whose weights are lifted.
    constexpr float kLift = kBF16 ? 0.f : 14.f, kSlack = kBF16 ? 8.f : 1.f;
    extern __shared__ __align__(128) uint8_t smem[];
    auto sum = reinterpret_cast<float (*)[kQ][D]>(smem);  // [kWarps][kQ][D], once the rings are done with
    static_assert(kWarps * kQ * D * 4 <= kSmem, "the sums fit where the rings were");
    __shared__ float warp_m[kWarps][kQ], warp_l[kWarps][kQ], cta_m[kQ], cta_l[kQ];

    wait_for_predecessor();
    if (a.parts > 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may be launched
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int share = a.H / a.HK, chunks = (share + kQ - 1) / kQ;
    const int rank = blockIdx.x % a.ranks, part = blockIdx.x / a.ranks % a.parts;
    const int row = blockIdx.x / a.ranks / a.parts;  // (sequence, key head, chunk of queries)
    const int chunk = row % chunks, kvh = row / chunks % a.HK, b = row / chunks / a.HK;
    const int first_q = kvh * share + chunk * kQ, queries = min(kQ, share - chunk * kQ);

    uint4 q[kGroups][kVec];
#pragma unroll
    for (int m = 0; m < kGroups; ++m)
#pragma unroll
        for (int c = 0; c < kVec; ++c)
            q[m][c] = 8 * m + g < queries ? *reinterpret_cast<const uint4 *>(
                                                a.Q + ((long long)b * a.H + first_q + 8 * m + g) * D + t * 8 + 32 * c)
                                          : make_uint4(0u, 0u, 0u, 0u);

    int len = a.lens[b], first = 0, entries = 0;
    if (a.row_ptr) {
        first = a.row_ptr[b];
        entries = a.row_ptr[b + 1] - first;
    }
    const int per_block = a.block / 16, cap = a.max_pages << a.page_shift, nb = (cap + a.block - 1) / a.block;
    if (len < 0 || len > cap) {
        if (tid == 0) raise_status(a.flags, kDevBadSchedule);
        len = 0;
    }
    if (a.row_ptr && (first < 0 || entries < 0 || entries > nb || first > a.nnz_cap - entries)) {
        if (tid == 0) raise_status(a.flags, kDevBadSchedule);
        entries = 0;
    }
    const int n16 = !a.row_ptr ? (len + 15) / 16 : len > 0 ? entries * per_block : 0;  // groups of 16 keys to visit
    const int workers = a.ranks * a.parts * kWarps, worker = (part * a.ranks + rank) * kWarps + warp;
    const int steps = (n16 + kSub - 1) / kSub;  // of all workers, dealt out in turn

    // Where group u of 16 keys begins, and its page; len (no keys) for what is not there.  (The page is asked
    // for before the length is known to reach it: a table's row has entries for all of `cap`.)
    auto place = [&](long long u, int &k0, int &page) {
        k0 = len;
        page = 0;
        long long k = u * 16;
        if (a.row_ptr) {
            if (u >= n16) return;
            const int e = (int)u / per_block, *entry = a.col_idx + first + e;
            const int j = *entry, before = e > 0 ? entry[-1] : -1;
            if (j < 0 || j >= nb || j <= before) {
                raise_status(a.flags, kDevBadSchedule);
                return;
            }
            k = (long long)j * a.block + u % per_block * 16;
        }
        if (k >= cap) return;
        const int p = a.page_table[(long long)b * a.max_pages + (k >> a.page_shift)];
        if (k >= len) return;
        if (p < 0 || p >= a.num_pages) {
            raise_status(a.flags, kDevBadSchedule);
            return;
        }
        k0 = (int)k;
        page = p;
    };
    // Lane i looks up group i % kSub of the warp's step kBatch * batch + i / kSub.
    auto places = [&](int batch, int &k0, int &page) {
        const long long step = worker + ((long long)batch * kBatch + lane / kSub) * workers;
        place(step * kSub + lane % kSub, k0, page);
    };
    const int mask = (1 << a.page_shift) - 1;
    const long long head_at = (long long)kvh << a.page_shift;
    auto row_at = [&](int k0, int page, int64_t page_stride) { return page * page_stride + (head_at + (k0 & mask)) * D; };

    int k0_now, page_now, k0_next = 0, page_next = 0;  // of this batch of steps, and the one after
    places(0, k0_now, page_now);
    // The copies of step n, 16 keys and then 16 values at a time, a group of copies in any case.
    const uint32_t ring = smem_u32(smem) + warp * kRing;
    constexpr int kPieces = D / 8, kRows = 32 / kPieces;  // pieces per row, rows that a warp's copy takes
    const int piece = lane % kPieces, row_in = lane / kPieces;
    auto copy_step = [&](int n, int batch) {
        const int at = n % kBatch;
        const bool now = n / kBatch == batch;
        const uint32_t to = ring + n % kStages * 2 * kHalf;
#pragma unroll
        for (int s = 0; s < kSub; ++s) {
            const int k0 = __shfl_sync(0xffffffffu, now ? k0_now : k0_next, at * kSub + s);
            const int page = __shfl_sync(0xffffffffu, now ? page_now : page_next, at * kSub + s);
            if (k0 >= len) {
#pragma unroll
                for (int i = 0; i < 16 / kRows; ++i) {
                    copy16(to + s * 2048 + i * 512 + lane * 16, a.K, false);
                    copy16(to + kHalf + s * 2048 + i * 512 + lane * 16, a.V, false);
                }
                continue;
            }
            const uint16_t *k = a.K + row_at(k0, page, a.k_page_stride) + lane * 8;
            const uint16_t *v = a.V + row_at(k0, page, a.v_page_stride) + lane * 8;
#pragma unroll
            for (int i = 0; i < 16 / kRows; ++i) {
                const int r = i * kRows + row_in;
                copy16(to + s * 2048 + r * 2 * D + ((piece ^ ((r & 1) << 2)) << 4), k + i * 256, k0 + r < len);
            }
#pragma unroll
            for (int i = 0; i < 16 / kRows; ++i) {
                const int r = i * kRows + row_in;
                copy16(to + kHalf + s * 2048 + r * 2 * D + ((piece ^ (r & 7)) << 4), v + i * 256, k0 + r < len);
            }
        }
    };
    const int mine = steps > worker ? (steps - worker + workers - 1) / workers : 0;  // this warp's steps
#pragma unroll
    for (int n = 0; n < kStages - 1; ++n) {
        if (n < mine) copy_step(n, 0);
        copies_begun();
    }
    if (mine > kBatch) places(1, k0_next, page_next);
    // a lane's pieces of a step's keys (rows g and g + 8), and its row of the values' 8 x 8 matrices (keys below 8,
    // then from 8 on; of two neighbouring pieces each)
    const uint32_t k_even = ring + g * 2 * D + ((t ^ ((g & 1) << 2)) << 4), k_odd = k_even ^ 64;
    const uint32_t v_row = ring + kHalf + ((lane & 7) + (lane >> 4) * 8) * 2 * D, v_piece = ((lane >> 3 & 1) ^ (lane & 7)) << 4;

    float m[kGroups][2], l[kGroups][2], acc[kGroups][kTiles][4];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
        m[i][0] = m[i][1] = -INFINITY;
        l[i][0] = l[i][1] = 0.f;
#pragma unroll
        for (int j = 0; j < kTiles; ++j) acc[i][j][0] = acc[i][j][1] = acc[i][j][2] = acc[i][j][3] = 0.f;
    }

    for (int n = 0; n < mine; ++n) {
        const int batch = n / kBatch;
        if (n > 0 && n % kBatch == 0) {
            k0_now = k0_next;
            page_now = page_next;
            if (mine > (batch + 1) * kBatch) places(batch + 1, k0_next, page_next);
        }
        if (n + kStages - 1 < mine) copy_step(n + kStages - 1, batch);
        copies_begun();
        copies_done<kStages - 1>();
        __syncwarp();
        const uint32_t stage = n % kStages * 2 * kHalf;
        float sc[kGroups][kSub][4];
#pragma unroll
        for (int s = 0; s < kSub; ++s) {
            float other[kGroups][4];  // half of the dimensions: two chains of products
#pragma unroll
            for (int i = 0; i < kGroups; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[i][s][e] = other[i][e] = 0.f;
#pragma unroll
            for (int v = 0; v < kVec; ++v) {
                const uint32_t at = (v & 1 ? k_odd : k_even) + stage + s * 2048 + v / 2 * 128;
                const uint4 x = load_piece(at), y = load_piece(at + 8 * 2 * D);
#pragma unroll
                for (int i = 0; i < kGroups; ++i) {
                    const uint4 &z = q[i][v];
                    mma<kBF16>(sc[i][s], x.x, y.x, x.y, y.y, z.x, z.y);
                    mma<kBF16>(other[i], x.z, y.z, x.w, y.w, z.z, z.w);
                }
            }
            const int k0 = __shfl_sync(0xffffffffu, k0_now, n % kBatch * kSub + s);
            const bool there = k0 + g < len, there8 = k0 + g + 8 < len;
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                float (&c)[4] = sc[i][s];
                c[0] = there ? (c[0] + other[i][0]) * a.scale_log2 : -INFINITY;
                c[1] = there ? (c[1] + other[i][1]) * a.scale_log2 : -INFINITY;
                c[2] = there8 ? (c[2] + other[i][2]) * a.scale_log2 : -INFINITY;
                c[3] = there8 ? (c[3] + other[i][3]) * a.scale_log2 : -INFINITY;
            }
        }
        // The reference of a query's weights follows its maximum only once a score is kSlack above it.
        bool grown = false;
        float top[kGroups][2];
#pragma unroll
        for (int i = 0; i < kGroups; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // queries 2 t and 2 t + 1
                top[i][e] = fmaxf(sc[i][0][e], sc[i][0][e + 2]);
#pragma unroll
                for (int s = 1; s < kSub; ++s) top[i][e] = fmaxf(top[i][e], fmaxf(sc[i][s][e], sc[i][s][e + 2]));
                grown |= top[i][e] > m[i][e] + kSlack;
            }
        if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
            for (int i = 0; i < kGroups; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float to = fmaxf(m[i][e], top[i][e]);
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, o));
                    const float keep = ex2_approx(m[i][e] - reference(to));
                    l[i][e] *= keep;
#pragma unroll
                    for (int j = 0; j < kTiles; ++j) {
                        acc[i][j][e] *= keep;
                        acc[i][j][e + 2] *= keep;
                    }
                    m[i][e] = to;
                }
        }
        uint32_t w[kGroups][kSub][2][kParts];
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            float p[kSub][4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float ref = reference(m[i][e]) - kLift;
#pragma unroll
                for (int s = 0; s < kSub; ++s) {
                    p[s][e] = ex2_approx(sc[i][s][e] - ref);
                    p[s][e + 2] = ex2_approx(sc[i][s][e + 2] - ref);
                    l[i][e] += p[s][e] + p[s][e + 2];
                }
            }
#pragma unroll
            for (int s = 0; s < kSub; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    in_parts<kBF16>(p[s][2 * h], p[s][2 * h + 1], w[i][s][h]);
#pragma unroll
                    for (uint32_t &x : w[i][s][h]) x = transpose8(x);
                }
        }
        // A tensor core rounds its sums towards 0, by up to 2^-23 of what they hold: a step's own sum is small, the smaller
        // products go first, and it is added to the row's rounded to the nearest.
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
            float step[kGroups][4];
#pragma unroll
            for (int i = 0; i < kGroups; ++i) step[i][0] = step[i][1] = step[i][2] = step[i][3] = 0.f;
#pragma unroll
            for (int s = 0; s < kSub; ++s) {
                uint32_t v[4];
                load_transposed(v_row + stage + s * 2048 + (v_piece ^ (j << 5 & 96)) + (j << 5 & ~96), v);
#pragma unroll
                for (int i = 0; i < kGroups; ++i)
#pragma unroll
                    for (int k = kParts - 1; k >= 0; --k)
                        mma<kBF16>(step[i], v[0], v[1], v[2], v[3], w[i][s][0][k], w[i][s][1][k]);
            }
#pragma unroll
            for (int i = 0; i < kGroups; ++i)
#pragma unroll
                for (int e = 0; e < 4; e += 2)
                    f2_unpack(f2_add(f2_pack(acc[i][j][e], acc[i][j][e + 1]), f2_pack(step[i][e], step[i][e + 1])), acc[i][j][e],
                              acc[i][j][e + 1]);
        }
        __syncwarp();  // the stage may be written again
    }

    // the warps' sums, then the cluster's
    copies_done<0>();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kGroups; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int query = 8 * i + 2 * t + e;
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], o);
            if (g == 0) {
                warp_m[warp][query] = m[i][e];
                warp_l[warp][query] = l[i][e];
            }
#pragma unroll
            for (int j = 0; j < kTiles; ++j) {
                sum[warp][query][16 * j + g] = acc[i][j][e];
                sum[warp][query][16 * j + g + 8] = acc[i][j][e + 2];
            }
        }
    __syncthreads();
    for (int at = tid; at < queries * D; at += kThreads) {
        const int query = at / D, d = at % D;
        float top = warp_m[0][query];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, warp_m[w][query]);
        float total = 0.f, y = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = ex2_approx(warp_m[w][query] - reference(top));
            total = fmaf(warp_l[w][query], f, total);
            y = fmaf(sum[w][query][d], f, y);
        }
        sum[0][query][d] = y;  // read by this thread alone so far
        if (d == 0) {
            cta_m[query] = top;
            cta_l[query] = total;
        }
    }
    if (a.ranks > 1) cluster_sync();
    else __syncthreads();
    for (int at = rank * kThreads + tid; at < queries * D; at += a.ranks * kThreads) {
        const int query = at / D, d = at % D;
        float top = -INFINITY, total = 0.f, y = 0.f;
        for (int r = 0; r < a.ranks; ++r) {
            const float m2 = a.ranks > 1 ? load_remote(&cta_m[query], r) : cta_m[query];
            const float l2 = a.ranks > 1 ? load_remote(&cta_l[query], r) : cta_l[query];
            const float y2 = a.ranks > 1 ? load_remote(&sum[0][query][d], r) : sum[0][query][d];
            const float mn = fmaxf(top, m2), f = ex2_approx(top - reference(mn)), f2 = ex2_approx(m2 - reference(mn));
            total = total * f + l2 * f2;
            y = y * f + y2 * f2;
            top = mn;
        }
        if (a.parts == 1) {
            // (a NaN among the scores is the answer's, too)
            store16<kBF16>(a.O + ((long long)b * a.H + first_q + query) * D + d, total == 0.f ? 0.f : y / total);
        } else {
            float *to = a.partial + (((long long)b * a.H + first_q + query) * a.parts + part) * (D + 2);
            to[d] = y;
            if (d == 0) {
                to[D] = top;
                to[D + 1] = total;
            }
        }
    }
    if (a.ranks > 1) cluster_sync();  // no thread block leaves while its shared memory may be read
}

// Joins the parts' sums of one query, D dimensions.  (Launched while the kernel that makes them still runs; it
// waits for all of that kernel before it reads.)
template <int D, bool kBF16>
__global__ void __launch_bounds__(D) join_parts_kernel(const float *partial, uint16_t *O, int parts) {
    wait_for_predecessor();
    const long long row = blockIdx.x;
    const int d = threadIdx.x;
    const float *from = partial + row * parts * (D + 2);
    float top = -INFINITY, total = 0.f, y = 0.f;
    for (int p = 0; p < parts; ++p, from += D + 2) {
        const float m2 = from[D], mn = fmaxf(top, m2);
        const float f = ex2_approx(top - reference(mn)), f2 = ex2_approx(m2 - reference(mn));
        total = total * f + from[D + 1] * f2;
        y = y * f + from[d] * f2;
        top = mn;
    }
    store16<kBF16>(O + row * D + d, total == 0.f ? 0.f : y / total);
}

int groups_of(const PagedDecodeLaunch &a) { return a.H / a.HK > 8 ? 2 : 1; }

template <int D, bool kBF16, int kGroups>
tsa_status launch_one(const PagedDecodeLaunch &a) {
    const int share = a.H / a.HK, chunks = (share + 8 * kGroups - 1) / (8 * kGroups);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)a.B * a.HK * chunks * a.parts * a.ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = a.stream;
    static std::atomic<unsigned long long> allowed{0};
    if (!allow_smem(allowed, reinterpret_cast<const void *>(paged_decode_kernel<D, kBF16, kGroups>), kSmem)) return TSA_ERR_CUDA;
    cudaLaunchAttribute attrs[2] = {{}, set_up_early()};
    attrs[0].id = cudaLaunchAttributeClusterDimension;
    attrs[0].val.clusterDim.x = (unsigned)a.ranks;
    attrs[0].val.clusterDim.y = attrs[0].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = 2;
    TSA_TRY(launched(cudaLaunchKernelEx(&cfg, paged_decode_kernel<D, kBF16, kGroups>, a)));
    if (a.parts > 1) {
        cudaLaunchConfig_t join = {};
        join.gridDim = dim3((unsigned)(a.B * a.H));
        join.blockDim = dim3(D);
        join.stream = a.stream;
        cudaLaunchAttribute early = set_up_early();
        join.attrs = &early;
        join.numAttrs = 1;
        TSA_TRY(launched(cudaLaunchKernelEx(&join, join_parts_kernel<D, kBF16>, (const float *)a.partial, a.O, a.parts)));
    }
    return TSA_OK;
}

template <int D, bool kBF16>
tsa_status launch_groups(const PagedDecodeLaunch &a) {
    return groups_of(a) == 1 ? launch_one<D, kBF16, 1>(a) : launch_one<D, kBF16, 2>(a);
}

}  // namespace

void split_paged_decode(PagedDecodeLaunch *a) {
    const int per = 8 * groups_of(*a), share = a->H / a->HK, kStep = a->D == 64 ? 32 : 16;
    const long long rows = (long long)a->B * a->HK * ((share + per - 1) / per);
    const long long cap = (long long)a->max_pages << a->page_shift;
    const long long keys = a->nnz_cap > 0 ? std::min(cap, ((long long)a->nnz_cap * a->block + a->B - 1) / a->B) : cap;
    const long long steps = (keys + kStep - 1) / kStep;  // of a row
    // Thread blocks per row.  As many as the GPU holds at once (two per multiprocessor, 32 clusters of eight)
    // while every warp has a step, clusters first: us with 1 / 2 / 4 / 8 of them, 16 rows of 32 steps 7.9 / 6.7 /
    // 5.2 / 5.3; 128 ragged rows of 86 steps 17.2 / 16.7 / 20.3 / 28.6 (all of one length 18.6 / 19.2 / 23.3 / 31.6); with
    // 1 / 4 clusters of eight, 8 rows of 8192 steps 139 / 83, of 256 steps 9.0 / 7.7.  Four times as many where each warp is
    // left 24 steps and the blocks would not fill their last wave, so that short and long rows even out: 256 ragged rows
    // of 384 steps 119 -> 110, 32 of 6000 steps, some empty, 206 -> 191 (none empty 257 -> 257); but 512 rows of 512 steps
    // 295 -> 297, 256 of 250 steps 83 -> 90 (ragged 63.3 -> 62.6).  Rows are taken as alike, and as long as the table is
    // wide: a long one among short ones has no more thread blocks than they.
    const long long slots = 2 * 152, clusters = 32;
    long long ranks = 1, parts = 1;
    while (ranks < 8 && 2 * ranks * rows <= slots && 2 * ranks * kWarps <= steps) ranks *= 2;
    if (ranks == 8) parts = std::max(1ll, std::min(clusters / rows, steps / (8 * kWarps * 2)));
    const long long blocks = rows * ranks * parts;
    if ((blocks <= slots || blocks % slots < slots / 2) && blocks < 4 * slots && steps >= 4 * ranks * parts * kWarps * 24)
        for (int i = 0; i < 2; ++i) (ranks < 8 ? ranks : parts) *= 2;
    a->ranks = (int)ranks;
    a->parts = (int)parts;
}

size_t paged_decode_workspace(const PagedDecodeLaunch &a) {
    return a.parts == 1 ? 0 : (size_t)a.B * a.H * a.parts * (a.D + 2) * sizeof(float);
}

tsa_status launch_paged_decode(const PagedDecodeLaunch &a) {
    if (a.D == 64) return a.bf16 ? launch_groups<64, true>(a) : launch_groups<64, false>(a);
    return a.bf16 ? launch_groups<128, true>(a) : launch_groups<128, false>(a);
}

}  // namespace tsa
