// decode.cu -- one new token per sequence against a key/value cache, with the score terms of
// score_terms.cuh: for sequence b of `len` tokens (the new one is the last, its key and value already
// in the cache) and every head, attention of the query at len - 1 over the keys of the cache blocks
// that row b of the schedule lists, z and the difference of maps as in the forward kernels.
//
// Bound by memory: each listed key and value row is read once, 4 D bytes per key and head, against
// 2 D multiply-adds (3 D with two maps), so the arithmetic stays on the FMA pipe.
//  * A lane of a warp holds 8 of the D dimensions, so D / 8 lanes read a row with one 16-byte load
//    each and a warp reads 2 (D = 128) or 4 rows per load.  A warp takes a chunk of 8 such loads of K
//    and 8 of V at a time (two maps: 4, to keep both sums in registers with 24 warps on an SM); the next
//    chunk's K is loaded while this one's V is used, so that 2 to 8 KB are in flight per warp at any time.
//  * Every group of D / 8 lanes keeps its own running maximum, denominator and 8 sums, in binary32;
//    the weights are never rounded.  They are joined at the end: groups by shuffles, warps through
//    shared memory, thread blocks through the shared memory of their cluster.
//  * The chunks of one (sequence, head) are dealt out to all warps of a cluster of thread blocks, so a
//    few long sequences fill the GPU as well as many short ones, with one launch, no workspace and a
//    join in a fixed order.
//  * A bias is one constant for a chunk beyond the last bucket's start; otherwise each lane finds the
//    bucket of one of the chunk's keys and the groups take theirs by a shuffle.
// Keys at len and beyond are neither read nor counted, so what the cache holds there does not matter.
// Measured, 16 sequences of 8192 tokens, 32 heads, D = 128, bf16, all blocks listed (2.15 GB): biased 316 us
// = 6.8 TB/s, differential 326 us = 6.6 TB/s; a copy reaches 6.8 TB/s, a kernel that only reads 7.0.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "score_terms.cuh"
#include "tsa_device.cuh"
#include "tsa_internal.h"

namespace tsa {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
// 16-byte loads of K (and of V) a lane has in flight: with two maps' sums to keep, half as many
template <class Terms>
constexpr int kLoadsOf = Terms::kDiff ? 4 : 8;

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// A float of thread block `rank`'s shared memory, at this thread block's address `p` of it.
__device__ __forceinline__ float load_remote(const float *p, uint32_t rank) {
    uint32_t at;
    float v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

template <bool kBF16>
__device__ __forceinline__ void widen8(const uint4 &w, float (&x)[8]) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        x[2 * t] = widen16<kBF16>(v[t] & 0xFFFFu);
        x[2 * t + 1] = kBF16 ? __uint_as_float(v[t] & 0xFFFF0000u) : widen16<kBF16>(v[t] >> 16);
    }
}

// One running softmax: the maximum (log2 units), the denominator and this lane's 8 sums.
struct Running {
    float m = -INFINITY, l = 0.f, acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};

    // The weights 2^(s - m) of the scores under the new maximum; what was there is rescaled.
    template <int kLoads>
    __device__ __forceinline__ void weigh(const float (&s)[kLoads], float (&p)[kLoads]) {
        float mx = m;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) mx = fmaxf(mx, s[i]);
        const float ref = mx == -INFINITY ? 0.f : mx;  // no key with weight yet
        if (mx > m) {
            const float keep = ex2_approx(m - ref);
            l *= keep;
#pragma unroll
            for (int d = 0; d < 8; ++d) acc[d] *= keep;
            m = mx;
        }
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            p[i] = ex2_approx(s[i] - ref);
            t += p[i];
        }
        l += t;
    }

    // Joins the state of the lane `off` away.
    __device__ __forceinline__ void join(int off) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, off), l2 = __shfl_xor_sync(0xffffffffu, l, off);
        const float mx = fmaxf(m, m2), ref = mx == -INFINITY ? 0.f : mx;
        const float a = ex2_approx(m - ref), b = ex2_approx(m2 - ref);
        l = l * a + l2 * b;
#pragma unroll
        for (int d = 0; d < 8; ++d) acc[d] = acc[d] * a + __shfl_xor_sync(0xffffffffu, acc[d], off) * b;
        m = mx;
    }
};

template <int D, bool kBF16, class Terms>
__global__ void __launch_bounds__(kThreads, Terms::kDiff ? 3 : 2)
decode_kernel(const uint16_t *__restrict__ Q, const uint16_t *__restrict__ K, const uint16_t *__restrict__ V,
              const int32_t *__restrict__ lens, const int32_t *__restrict__ row_ptr,
              const int32_t *__restrict__ col_idx, int nnz_cap, uint16_t *__restrict__ O, int H, int cap, int block,
              float scale_log2, DeviceFlags flags, const __grid_constant__ Terms terms) {
    constexpr bool kBias = Terms::kBias, kDiff = Terms::kDiff;
    constexpr int kMaps = kDiff ? 2 : 1, kLoads = kLoadsOf<Terms>;
    constexpr int kG = D / 8;            // lanes per row
    constexpr int kPer = 32 / kG;        // rows per load of a warp
    constexpr int kChunk = kLoads * kPer;
    __shared__ __align__(16) float warp_acc[kMaps][kWarps][D];
    __shared__ float warp_m[kMaps][kWarps], warp_l[kMaps][kWarps];
    __shared__ float cta_m[kMaps], cta_l[kMaps], cta_acc[kMaps][D];
    __shared__ __align__(16) uint8_t table_smem[kBias ? kBucketBytes : 16];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ranks = (int)cluster_size(), rank = (int)cluster_rank();
    const long long at = blockIdx.x / ranks;  // sequence * H + head
    const int b = (int)(at / H), head = (int)(at % H);
    const int group = lane / kG, li = lane % kG;

    [[maybe_unused]] const BucketTable table(table_smem);
    if constexpr (kBias) {
        table.template load<kBF16>(terms, head, tid, kThreads);
        __syncthreads();
    }
    [[maybe_unused]] float lam = 0.f;
    if constexpr (kDiff) lam = lambda_of<D / 2, kBF16>(terms, head);

    const int nb = (cap + block - 1) / block;
    int len = __ldg(lens + b), first = __ldg(row_ptr + b), entries = __ldg(row_ptr + b + 1) - first;
    const bool bad_len = len < 0 || len > cap;
    if (bad_len || first < 0 || entries < 0 || entries > nb || first > nnz_cap - entries) {
        if (tid == 0) raise_status(flags, kDevBadSchedule);
        entries = 0;
    }
    float q[8];
    widen8<kBF16>(__ldg(reinterpret_cast<const uint4 *>(Q + at * D) + li), q);
#pragma unroll
    for (int d = 0; d < 8; ++d) q[d] *= scale_log2;
    const uint16_t *Kl = K + at * cap * D + li * 8, *Vl = V + at * cap * D + li * 8;

    Running state[kMaps];
    const int per_block = block / kChunk, chunks = entries * per_block, step = ranks * kWarps;
    // The block of chunk u and the one listed before it (entries past the end: none).
    auto entry_of = [&](int u, int &j, int &before) {
        j = before = -1;
        if (u < chunks) {
            const int *at_entry = col_idx + first + u / per_block;
            j = __ldg(at_entry);
            if (u >= per_block) before = __ldg(at_entry - 1);
        }
    };
    // First key of chunk u; len (a chunk without keys) for a block outside the cache or out of order.
    auto first_key = [&](int u, int j, int before) {
        if (u >= chunks) return len;
        if (j >= nb || j <= before || j < 0) {
            if (lane == 0) raise_status(flags, kDevBadSchedule);
            return len;
        }
        return j * block + (u % per_block) * kChunk;
    };
    auto load = [&](uint4 (&r)[kLoads], const uint16_t *base, int k0) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int k = k0 + i * kPer + group;
            r[i] = k < len ? __ldg(reinterpret_cast<const uint4 *>(base + (long long)k * D)) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    // K of a chunk is loaded while the one before is weighed, V while its scores are summed: a warp
    // always has a chunk's rows in flight.
    int u = rank * kWarps + warp, j, before;
    entry_of(u, j, before);
    int k0 = first_key(u, j, before);
    uint4 kr[kLoads], vr[kLoads];
    load(kr, Kl, k0);
    entry_of(u + step, j, before);
    for (; u < chunks; u += step) {
        load(vr, Vl, k0);
        // the bias of chunk key `lane`, or of all of them
        [[maybe_unused]] float mine = 0.f;
        [[maybe_unused]] bool uniform = true;
        if constexpr (kBias) {
            const int last = terms.n - 1;
            uniform = len - k0 - kChunk >= table.start[last];  // the nearest key's distance
            mine = table.bias[last];
            if (!uniform) {
                const int d = max(len - 1 - k0 - lane, 0);
                int lo = 0, hi = last;  // the last bucket that starts at or before d
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (table.start[mid] <= d) lo = mid;
                    else hi = mid - 1;
                }
                mine = table.bias[lo];
            }
        }
        float s[kMaps][kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            float x[8];
            uint64_t two = f2_pack(0.f, 0.f);
            widen8<kBF16>(kr[i], x);
#pragma unroll
            for (int d = 0; d < 8; d += 2)
                two = f2_fma(f2_pack(q[d], q[d + 1]), f2_pack(x[d], x[d + 1]), two);
            float dot, odd;
            f2_unpack(two, dot, odd);
            dot += odd;
#pragma unroll
            for (int o = 1; o < kG / kMaps; o <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
            const bool there = k0 + i * kPer + group < len;
            if constexpr (kDiff) {
                const float other = __shfl_xor_sync(0xffffffffu, dot, kG / 2);
                s[0][i] = there ? (li < kG / 2 ? dot : other) : -INFINITY;
                s[1][i] = there ? (li < kG / 2 ? other : dot) : -INFINITY;
            } else {
                if constexpr (kBias) {
                    const float one = __shfl_sync(0xffffffffu, mine, i * kPer + group);
                    dot += uniform ? mine : one;
                }
                s[0][i] = there ? dot : -INFINITY;
            }
        }
        const int next = first_key(u + step, j, before);
        load(kr, Kl, next);
        entry_of(u + 2 * step, j, before);
        float p[kMaps][kLoads];
#pragma unroll
        for (int m = 0; m < kMaps; ++m) state[m].weigh(s[m], p[m]);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            float x[8];
            widen8<kBF16>(vr[i], x);
#pragma unroll
            for (int m = 0; m < kMaps; ++m)
#pragma unroll
                for (int d = 0; d < 8; d += 2)
                    f2_unpack(f2_fma(f2_pack(p[m][i], p[m][i]), f2_pack(x[d], x[d + 1]),
                                     f2_pack(state[m].acc[d], state[m].acc[d + 1])),
                              state[m].acc[d], state[m].acc[d + 1]);
        }
        k0 = next;
    }
    // groups of a warp, then the warps
#pragma unroll
    for (int m = 0; m < kMaps; ++m) {
#pragma unroll
        for (int o = kG; o < 32; o <<= 1) state[m].join(o);
        if (lane == 0) {
            warp_m[m][warp] = state[m].m;
            warp_l[m][warp] = state[m].l;
        }
        if (group == 0) {
            float4 *to = reinterpret_cast<float4 *>(&warp_acc[m][warp][li * 8]);
            to[0] = make_float4(state[m].acc[0], state[m].acc[1], state[m].acc[2], state[m].acc[3]);
            to[1] = make_float4(state[m].acc[4], state[m].acc[5], state[m].acc[6], state[m].acc[7]);
        }
    }
    __syncthreads();
    if (tid < D) {
#pragma unroll
        for (int m = 0; m < kMaps; ++m) {
            float mx = warp_m[m][0];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, warp_m[m][w]);
            const float ref = mx == -INFINITY ? 0.f : mx;
            float l = 0.f, a = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2_approx(warp_m[m][w] - ref);
                l = fmaf(warp_l[m][w], f, l);
                a = fmaf(warp_acc[m][w][tid], f, a);
            }
            cta_acc[m][tid] = a;
            if (tid == 0) {
                cta_m[m] = mx;
                cta_l[m] = l;
            }
        }
    }
    cluster_sync();
    if (rank == 0 && tid < D) {
        float o[kMaps];
#pragma unroll
        for (int m = 0; m < kMaps; ++m) {
            float mx = cta_m[m], l = cta_l[m], a = cta_acc[m][tid];
            for (int r = 1; r < ranks; ++r) {
                const float m2 = load_remote(&cta_m[m], r), l2 = load_remote(&cta_l[m], r),
                            a2 = load_remote(&cta_acc[m][tid], r);
                const float mn = fmaxf(mx, m2), ref = mn == -INFINITY ? 0.f : mn;
                const float f = ex2_approx(mx - ref), f2 = ex2_approx(m2 - ref);
                l = l * f + l2 * f2;
                a = a * f + a2 * f2;
                mx = mn;
            }
            o[m] = l == 0.f ? 0.f : a / l;  // (a NaN among the scores is the answer's, too)
        }
        float y = o[0];
        if constexpr (kDiff) y = fmaf(-lam, o[1], o[0]);
        if constexpr (kBF16) O[at * D + tid] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
        else O[at * D + tid] = __half_as_ushort(__float2half_rn(y));
    }
    cluster_sync();  // no thread block leaves while its shared memory may be read
}

template <int D, bool kBF16, class Terms>
tsa_status launch_one(const DecodeLaunch &a, const Terms &terms) {
    // Thread blocks per (sequence, head), up to a cluster of 8: as many as leave every warp a chunk of an
    // average row (the host knows no single row's length) while the GPU holds them all, and beyond that as
    // many as leave it 32 chunks, since each block pays for its start and its join.  us with 1 / 2 / 4 / 8
    // blocks (D = 128; biased, differential): 8 heads, rows of 128 blocks 73 / 40 / 23 / 14 and 115 / 61 / 35 /
    // 21; 128 heads, 13 blocks 11.4 / 10.1 / 13.8 / 21.0 and 15.6 / 13.8 / 17.6 / 23.8; 512 heads, 42 blocks
    // 108 / 116 / 117 / 147 and 148 / 127 / 128 / 157; 512 heads, ragged to 128 blocks 267 / 247 / 243 / 263
    // and 330 / 289 / 273 / 302.
    constexpr int kChunk = kLoadsOf<Terms> * 32 / (D / 8);
    const long long sequences = a.lanes / a.H;
    const long long row = std::min((long long)a.cap, ((long long)a.nnz_cap * a.block + sequences - 1) / sequences);
    const long long chunks = (row + kChunk - 1) / kChunk;
    const long long slots = (long long)a.sms * (Terms::kDiff ? 3 : 2);  // thread blocks that run at once
    unsigned ranks = 1;
    while (ranks < 8) {
        const long long least = 2 * ranks * (long long)a.lanes <= slots ? 1 : 32;
        if (ranks * kWarps * least >= chunks) break;
        ranks *= 2;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.lanes * ranks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = a.stream;
    cudaLaunchAttribute cluster;
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = ranks;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    cfg.attrs = &cluster;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, decode_kernel<D, kBF16, Terms>, a.Q, a.K, a.V, a.lens, a.row_ptr, a.col_idx,
                              a.nnz_cap, a.O, a.H, a.cap, a.block, a.scale_log2, a.flags, terms) == cudaSuccess
               ? TSA_OK
               : TSA_ERR_CUDA;
}

template <class Terms>
tsa_status launch(const DecodeLaunch &a, const Terms &terms) {
    if (a.D == 64) return a.bf16 ? launch_one<64, true>(a, terms) : launch_one<64, false>(a, terms);
    if (a.D == 128) return a.bf16 ? launch_one<128, true>(a, terms) : launch_one<128, false>(a, terms);
    return TSA_ERR_UNSUPPORTED;
}

}  // namespace

tsa_status launch_biased_decode(const DecodeLaunch &a, const BiasTerms &terms) { return launch(a, terms); }
tsa_status launch_differential_decode(const DecodeLaunch &a, const DiffTerms &terms) { return launch(a, terms); }

}  // namespace tsa
