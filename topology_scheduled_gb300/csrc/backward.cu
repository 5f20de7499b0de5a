// backward.cu -- gradients of the scheduled causal attention on tcgen05 tensor cores (sm_103a).
//
// The forward is the kernel of "Add topology-derived sparse attention kernel"
// (triton-lang/kernels#22, Summary); its mirror page's segment-boundary record notes that the
// merged kernel has no backward pass, which is the step this file adds.  With P the softmax of
// the scaled scores over each query's allowed keys (the CSR row's blocks, keys <= the query in
// the diagonal block) and dO the upstream gradient:
//   Delta_q = <dO_q, O_q>,  dP = dO V^T,  dS = P o (dP - Delta),
//   dV = P^T dO,  dQ = scale dS K,  dK = scale dS^T Q.
// P is recomputed from the forward's log-sum-exp (P = exp(scale s - lse)), so nothing of size
// S x S is stored.
//
// Launches:
//   bwd_rows, bwd_col_count, bwd_col_scan, bwd_col_fill -- the transposed schedule: for every
//     key block j the ascending list of query blocks whose row holds j (a column bitmap, so
//     the lists come out sorted without a sort); rows are checked on the way (a row is cut at
//     its first entry that is out of order or out of [0, i], and the status word reports it).
//   bwd_delta -- Delta per query row from the stored O and dO.
//   bwd_dq_kernel -- one CTA per pair of query blocks (M = 128), walking the union of the two
//     CSR rows like the forward: S = Q K^T and dP = dO V^T into TMEM, dS formed by the
//     elementwise warps and written back over S in the input dtype, dQ += dS K with dS read
//     from TMEM.
//   bwd_dkv_kernel -- one CTA per pair of key blocks (M = 128), walking the union of the two
//     transposed columns: S^T = K Q^T and dP^T = V dO^T into TMEM, P^T and dS^T written back
//     over them, dV += P^T dO and dK += dS^T Q.
// Warp roles are those of the forward: one warp produces (TMA, rings of four blocks), one issues the
// MMAs from one thread (the next step's products before the current step's accumulation), and eight do
// the elementwise work, two per 32 rows with 32 columns of a step each (no value of a row is needed by
// the other).  A partial last block (S not a multiple of 64) needs no code of its own: the maps see
// [lanes, S, D] as three dimensions, so rows past a lane's end read as zero, whatever the next lane
// holds, and are not written.  Every wait is bounded; on a timeout a CTA records TSA_ERR_TIMEOUT, drains what it
// issued, frees its TMEM and returns.
#include "backward_kernels.cuh"

namespace tsa {
namespace {

// ---------------------------------------------------------------- transposed schedule

// One warp per CSR row: the valid prefix length (0 when it does not lie in [0, cap)), and bit i of
// column j's bitmap words for each valid entry j of row i.
__global__ void bwd_rows(int nb, const int32_t *__restrict__ row_ptr, const int32_t *__restrict__ col_idx,
                         long long cap, int words, int *__restrict__ vlen, unsigned *__restrict__ bitmap,
                         DeviceFlags flags) {
    const int lane = threadIdx.x & 31;
    const int nw = gridDim.x * (blockDim.x >> 5);
    for (int i = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); i < nb; i += nw) {
        const int b = row_ptr[i], len = row_ptr[i + 1] - b;
        int valid = 0;
        if (len >= 0 && len <= i + 1 && b >= 0 && (long long)b + len <= cap) {
            valid = len;
            for (int e0 = 0; e0 < len; e0 += 32) {
                const int e = e0 + lane;
                bool bad = false;
                if (e < len) {
                    const int j = col_idx[b + e];
                    const int prev = e > 0 ? col_idx[b + e - 1] : -1;
                    bad = j < 0 || j > i || j <= prev;
                }
                const unsigned m = __ballot_sync(0xffffffffu, bad);
                if (m) {
                    valid = e0 + __ffs(m) - 1;
                    break;
                }
            }
        }
        if (lane == 0 && valid != len) raise_status(flags, kDevBadSchedule);
        for (int e = lane; e < valid; e += 32) {
            const int j = col_idx[b + e];
            atomicOr(&bitmap[(size_t)j * words + (i >> 5)], 1u << (i & 31));
        }
        if (lane == 0) vlen[i] = valid;
    }
}

// A CSR of 128-token blocks as the CSR of 64-token blocks with the same allowed keys: query
// block a = 2p + h (64 tokens) of 128-block row p holds the 64-blocks 2j and 2j+1 of every
// j < p in row p, and of j = p the ones not after it (2p; 2p+1 when h = 1) -- the token mask
// of the 64-token diagonal block then cuts keys k > q exactly as the 128-token rule does.
// One warp per 128-block row: its valid prefix (the checks of bwd_rows), the two counts.
__global__ void bwd_expand128_count(int nb128, int nb64, const int32_t *__restrict__ row_ptr,
                                    const int32_t *__restrict__ col_idx, long long cap, int *__restrict__ vlen128,
                                    int *__restrict__ cnt64, DeviceFlags flags) {
    const int lane = threadIdx.x & 31;
    const int nw = gridDim.x * (blockDim.x >> 5);
    for (int p = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); p < nb128; p += nw) {
        const int b = row_ptr[p], len = row_ptr[p + 1] - b;
        int valid = 0;
        if (len >= 0 && len <= p + 1 && b >= 0 && (long long)b + len <= cap) {
            valid = len;
            for (int e0 = 0; e0 < len; e0 += 32) {
                const int e = e0 + lane;
                bool bad = false;
                if (e < len) {
                    const int j = col_idx[b + e];
                    const int prev = e > 0 ? col_idx[b + e - 1] : -1;
                    bad = j < 0 || j > p || j <= prev;
                }
                const unsigned m = __ballot_sync(0xffffffffu, bad);
                if (m) {
                    valid = e0 + __ffs(m) - 1;
                    break;
                }
            }
        }
        if (lane == 0) {
            if (valid != len) raise_status(flags, kDevBadSchedule);
            const int diag = valid > 0 && col_idx[b + valid - 1] == p ? 1 : 0;
            const int below = valid - diag;
            vlen128[p] = valid;
            cnt64[2 * p] = 2 * below + diag;
            if (2 * p + 1 < nb64) cnt64[2 * p + 1] = 2 * below + 2 * diag;
        }
    }
}

// One warp per 128-block row: writes the two 64-token rows at the scanned offsets.
__global__ void bwd_expand128_fill(int nb128, int nb64, const int32_t *__restrict__ row_ptr,
                                   const int32_t *__restrict__ col_idx, const int *__restrict__ vlen128,
                                   const int *__restrict__ rp64, int32_t *__restrict__ ci64) {
    const int lane = threadIdx.x & 31;
    const int nw = gridDim.x * (blockDim.x >> 5);
    for (int p = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); p < nb128; p += nw) {
        const int b = row_ptr[p], valid = vlen128[p];
        const bool second = 2 * p + 1 < nb64;
        // an overflowing total leaves the offsets equal (every row empty): nothing to write
        const int o0 = rp64[2 * p], o1 = second ? rp64[2 * p + 1] : 0;
        const bool room0 = rp64[2 * p + 1] > o0 || valid == 0;
        const bool room1 = second && (rp64[2 * p + 2] > o1 || valid == 0);
        for (int e = lane; e < valid; e += 32) {
            const int j = col_idx[b + e];
            if (j < p) {
                if (room0) { ci64[o0 + 2 * e] = 2 * j; ci64[o0 + 2 * e + 1] = 2 * j + 1; }
                if (room1) { ci64[o1 + 2 * e] = 2 * j; ci64[o1 + 2 * e + 1] = 2 * j + 1; }
            } else {  // j == p, the last entry
                if (room0) ci64[o0 + 2 * e] = 2 * p;
                if (room1) { ci64[o1 + 2 * e] = 2 * p; ci64[o1 + 2 * e + 1] = 2 * p + 1; }
            }
        }
    }
}

// One warp per column: number of query blocks whose row holds it.
__global__ void bwd_col_count(int nb, int words, const unsigned *__restrict__ bitmap, int *__restrict__ cnt) {
    const int lane = threadIdx.x & 31;
    const int nw = gridDim.x * (blockDim.x >> 5);
    for (int j = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); j < nb; j += nw) {
        int c = 0;
        for (int w = lane; w < words; w += 32) c += __popc(bitmap[(size_t)j * words + w]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) c += __shfl_xor_sync(0xffffffffu, c, off);
        if (lane == 0) cnt[j] = c;
    }
}

// One CTA: col_ptr = exclusive scan of the counts.  If the total exceeds the capacity of the
// row list, every column is left empty and the status word reports it.
__global__ void __launch_bounds__(1024) bwd_col_scan(int nb, const int *__restrict__ cnt, int *__restrict__ col_ptr,
                                                     long long cap, DeviceFlags flags) {
    __shared__ long long warp_tot[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nwarps = blockDim.x >> 5;
    const int per = (nb + blockDim.x - 1) / blockDim.x;
    const int beg = min(nb, tid * per), end = min(nb, beg + per);
    long long run = 0;
    for (int j = beg; j < end; ++j) run += cnt[j];
    long long incl = run;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
    }
    if (lane == 31) warp_tot[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        long long t = lane < nwarps ? warp_tot[lane] : 0;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, t, off);
            if (lane >= off) t += o;
        }
        warp_tot[lane] = t;
    }
    __syncthreads();
    const long long total = warp_tot[nwarps - 1];
    const bool fits = total <= cap;
    long long at = (warp > 0 ? warp_tot[warp - 1] : 0) + incl - run;
    for (int j = beg; j < end; ++j) {
        col_ptr[j] = fits ? (int)at : 0;
        at += cnt[j];
    }
    if (tid == 0) {
        col_ptr[nb] = fits ? (int)total : 0;
        if (!fits) raise_status(flags, kDevCapacity);
    }
}

// One warp per column: its query blocks in ascending order.
__global__ void bwd_col_fill(int nb, int words, const unsigned *__restrict__ bitmap,
                             const int *__restrict__ col_ptr, int32_t *__restrict__ row_idx) {
    const int lane = threadIdx.x & 31;
    const int nw = gridDim.x * (blockDim.x >> 5);
    for (int j = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); j < nb; j += nw) {
        int off = col_ptr[j];
        const int end = col_ptr[j + 1];
        for (int w0 = 0; w0 < words; w0 += 32) {
            const int w = w0 + lane;
            unsigned bits = w < words ? bitmap[(size_t)j * words + w] : 0u;
            const int c = __popc(bits);
            int incl = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += x;
            }
            int pos = off + incl - c;
            while (bits) {
                const int bit = __ffs(bits) - 1;
                if (pos < end) row_idx[pos] = w * 32 + bit;
                ++pos;
                bits &= bits - 1u;
            }
            off += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
}

// One CTA: the key blocks sorted by the length of their transposed column (descending, then
// by index) and paired in that order -- pairs[2p], pairs[2p+1] (-1 if nb is odd and p is the
// last pair).  A dK/dV CTA walks the union of its two columns, so pairing a long column (a
// sink or top-k block that nearly every query block holds) with a short one would leave half
// of its 128-row tile idle for the whole long walk; sorted pairs also put the longest walks
// first in launch order.  Bitonic sort of (~count << 32 | j) keys in shared memory.
__global__ void __launch_bounds__(1024) bwd_col_pairs(int nb, int pow2, const int *__restrict__ cnt,
                                                       int *__restrict__ pairs) {
    extern __shared__ unsigned long long keys[];
    for (int i = threadIdx.x; i < pow2; i += blockDim.x)
        keys[i] = i < nb ? ((unsigned long long)(0xFFFFFFFFu - (unsigned)cnt[i]) << 32) | (unsigned)i : ~0ull;
    __syncthreads();
    for (int k = 2; k <= pow2; k <<= 1) {
        for (int j = k >> 1; j > 0; j >>= 1) {
            for (int i = threadIdx.x; i < pow2; i += blockDim.x) {
                const int p = i ^ j;
                if (p > i) {
                    const unsigned long long a = keys[i], b = keys[p];
                    if ((a > b) == ((i & k) == 0)) {
                        keys[i] = b;
                        keys[p] = a;
                    }
                }
            }
            __syncthreads();
        }
    }
    const int npairs = (nb + 1) >> 1;
    for (int q = threadIdx.x; q < 2 * npairs; q += blockDim.x)
        pairs[q] = q < nb ? (int)(keys[q] & 0xFFFFFFFFull) : -1;
}

// ---------------------------------------------------------------- Delta = rowsum(dO * O)
// Delta per row in fp32.  kG = D / 8 threads per row (8 or 16, so a row never straddles a warp),
// each reading 16 bytes of O and of dO; products summed in the thread, then across the group.
// Grid: y over lanes, x over a lane's (row, 16-byte chunk) items -- at most 8192 * 64 * 16, so
// 32-bit indices and shifts -- with four items per thread whose loads are all issued before
// their arithmetic.  Rows are laid out per lane over Sp = nb * 64 tokens; the tokens past S (a
// partial last block) get Delta 0 and log-sum-exp +inf (see padded_lse), and the given log-sum-exp
// is copied into the same layout.
constexpr int kDeltaItems = 4;
template <bool kBF16, int kG>
__global__ void __launch_bounds__(256) bwd_delta(const uint16_t *__restrict__ O, const uint16_t *__restrict__ dO,
                                                 const float *__restrict__ lse, int S, int Sp,
                                                 float *__restrict__ delta, float *__restrict__ lse_pad,
                                                 const __grid_constant__ SmallSchedule schedule) {
    if (schedule.nb > 0 && blockIdx.x == gridDim.x - 1) {  // one block more per lane; the first lane's works
        if (blockIdx.y == 0) build_small_schedule(schedule);
        return;
    }
    constexpr int D = kG * 8;
    const long long lane = blockIdx.y;
    const int per_lane = Sp * kG;
    const int first = (int)blockIdx.x * (int)blockDim.x * kDeltaItems + (int)threadIdx.x;
    uint4 a[kDeltaItems], b[kDeltaItems];
#pragma unroll
    for (int k = 0; k < kDeltaItems; ++k) {
        const int x = first + k * (int)blockDim.x;
        const int t = x / kG;  // token within the lane
        if (x < per_lane && t < S) {
            const size_t off = (size_t)(lane * S + t) * D + (size_t)(x % kG) * 8;
            a[k] = __ldg(reinterpret_cast<const uint4 *>(O + off));
            b[k] = __ldg(reinterpret_cast<const uint4 *>(dO + off));
        } else {
            a[k] = b[k] = make_uint4(0u, 0u, 0u, 0u);
        }
    }
#pragma unroll
    for (int k = 0; k < kDeltaItems; ++k) {
        const int x = first + k * (int)blockDim.x;
        const int t = x / kG;
        const uint32_t av[4] = {a[k].x, a[k].y, a[k].z, a[k].w}, bv[4] = {b[k].x, b[k].y, b[k].z, b[k].w};
        float acc = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            acc = fmaf(widen16<kBF16>(av[q] & 0xFFFFu), widen16<kBF16>(bv[q] & 0xFFFFu), acc);
            acc = fmaf(widen16<kBF16>(av[q] >> 16), widen16<kBF16>(bv[q] >> 16), acc);
        }
#pragma unroll
        for (int off = kG >> 1; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
        if (x < per_lane && x % kG == 0) {
            const long long pr = lane * Sp + t;  // padded row
            delta[pr] = acc;
            lse_pad[pr] = t < S ? padded_lse(__ldg(lse + lane * S + t)) : INFINITY;
        }
    }
}

}  // namespace

BwdWorkspace backward_workspace_layout(int64_t lanes, int64_t S, int64_t nb, int64_t nnz_cap, int64_t nb_in) {
    BwdWorkspace w{};
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o = (o + bytes + 255) & ~(size_t)255;
        return at;
    };
    const int64_t words = (nb + 31) / 32;
    w.delta = take(sizeof(float) * (size_t)(lanes * nb * 64));  // rows padded to whole blocks
    w.lse_pad = take(sizeof(float) * (size_t)(lanes * nb * 64));
    w.vlen = take(sizeof(int) * (size_t)nb);
    w.cnt = take(sizeof(int) * (size_t)nb);
    w.col_ptr = take(sizeof(int) * (size_t)(nb + 1));
    w.bitmap = take(sizeof(unsigned) * (size_t)(nb * words));
    w.bitmap_bytes = sizeof(unsigned) * (size_t)(nb * words);
    w.row_idx = take(sizeof(int32_t) * (size_t)(nnz_cap > 0 ? nnz_cap : 1));
    w.pairs = take(sizeof(int) * (size_t)(2 * ((nb + 1) / 2)));
    // a CSR of 128-token blocks (nb_in rows) expanded to 64-token blocks: nnz_cap is then the
    // expanded capacity
    w.vlen_in = take(sizeof(int) * (size_t)(nb_in > 0 ? nb_in : 1));
    w.rp64 = take(sizeof(int32_t) * (size_t)(nb + 1));
    w.ci64 = take(sizeof(int32_t) * (size_t)(nb_in > 0 ? nnz_cap : 1));
    w.total = o;
    return w;
}

SmallSchedule small_schedule(const BwdLaunch &a) {
    SmallSchedule g{};
    if (a.nb_in > 0 || a.nb > kSmallBlocks) return g;
    g.nb = a.nb;
    g.row_ptr = a.row_ptr;
    g.col_idx = a.col_idx;
    g.read_cap = a.read_cap;
    g.cap = a.nnz_cap;
    g.vlen = a.vlen;
    g.col_ptr = a.col_ptr;
    g.pairs = a.pairs;
    g.row_idx = a.row_idx;
    g.flags = a.flags;
    return g;
}

tsa_status launch_backward_schedule(BwdLaunch *launch) {
    BwdLaunch &a = *launch;
    if (small_schedule(a).nb > 0) return TSA_OK;  // built beside Delta
    cudaStream_t st = a.stream;
    const int nb = a.nb;
    const int words = (nb + 31) / 32;
    const unsigned wgrid = (unsigned)((nb + 7) / 8 < 152 * 8 ? (nb + 7) / 8 : 152 * 8);
    if (a.nb_in > 0) {
        // 128-token CSR: the equivalent 64-token CSR first (cnt is free until the columns)
        const unsigned g = (unsigned)((a.nb_in + 7) / 8 < 152 * 8 ? (a.nb_in + 7) / 8 : 152 * 8);
        bwd_expand128_count<<<g, 256, 0, st>>>(a.nb_in, nb, a.row_ptr, a.col_idx, a.read_cap, a.vlen_in, a.cnt, a.flags);
        bwd_col_scan<<<1, 1024, 0, st>>>(nb, a.cnt, a.rp64, (long long)a.nnz_cap, a.flags);
        bwd_expand128_fill<<<g, 256, 0, st>>>(a.nb_in, nb, a.row_ptr, a.col_idx, a.vlen_in, a.rp64, a.ci64);
        a.row_ptr = a.rp64;
        a.col_idx = a.ci64;
        a.read_cap = a.nnz_cap;
    }
    if (cudaMemsetAsync(a.bitmap, 0, a.bitmap_bytes, st) != cudaSuccess) return TSA_ERR_CUDA;
    bwd_rows<<<wgrid, 256, 0, st>>>(nb, a.row_ptr, a.col_idx, a.read_cap, words, a.vlen, a.bitmap, a.flags);
    bwd_col_count<<<wgrid, 256, 0, st>>>(nb, words, a.bitmap, a.cnt);
    bwd_col_scan<<<1, 1024, 0, st>>>(nb, a.cnt, a.col_ptr, (long long)a.nnz_cap, a.flags);
    bwd_col_fill<<<wgrid, 256, 0, st>>>(nb, words, a.bitmap, a.col_ptr, a.row_idx);
    {
        int pow2 = 1;
        while (pow2 < nb) pow2 <<= 1;
        const size_t smem = sizeof(unsigned long long) * (size_t)pow2;
        // (the limit is the kernel's, not the call's: always the most that any call needs, so that no call
        // on another thread lowers it before this launch)
        static std::atomic<unsigned long long> ready{0};
        constexpr int kMost = (int)(sizeof(unsigned long long) * kMaxBackwardBlocks);
        if (!allow_smem(ready, reinterpret_cast<const void *>(bwd_col_pairs), kMost)) return TSA_ERR_CUDA;
        bwd_col_pairs<<<1, 1024, smem, st>>>(nb, pow2, a.cnt, a.pairs);
    }
    return cudaGetLastError() == cudaSuccess ? TSA_OK : TSA_ERR_CUDA;
}

tsa_status launch_backward_delta(const BwdLaunch &a) {
    cudaStream_t st = a.stream;
    const int Sp = a.nb * kBlock;
    const int per_lane = Sp * (a.D / 8);
    const SmallSchedule g = small_schedule(a);
    const dim3 grid((unsigned)((per_lane + 256 * kDeltaItems - 1) / (256 * kDeltaItems)) + (g.nb > 0 ? 1u : 0u),
                    (unsigned)a.lanes);
    if (a.D == 128) {
        if (a.bf16) bwd_delta<true, 16><<<grid, 256, 0, st>>>(a.O, a.dO, a.lse, a.S, Sp, a.delta, a.lse_pad, g);
        else bwd_delta<false, 16><<<grid, 256, 0, st>>>(a.O, a.dO, a.lse, a.S, Sp, a.delta, a.lse_pad, g);
    } else if (a.D == 64) {
        if (a.bf16) bwd_delta<true, 8><<<grid, 256, 0, st>>>(a.O, a.dO, a.lse, a.S, Sp, a.delta, a.lse_pad, g);
        else bwd_delta<false, 8><<<grid, 256, 0, st>>>(a.O, a.dO, a.lse, a.S, Sp, a.delta, a.lse_pad, g);
    } else {
        return TSA_ERR_UNSUPPORTED;
    }
    return cudaGetLastError() == cudaSuccess ? TSA_OK : TSA_ERR_CUDA;
}

tsa_status launch_attention_backward(const BwdLaunch &a_in) {
    BwdLaunch a = a_in;
    TSA_TRY(launch_backward_schedule(&a));
    TSA_TRY(launch_backward_delta(a));
    return launch_gradients(a, NoTerms{});
}

}  // namespace tsa
