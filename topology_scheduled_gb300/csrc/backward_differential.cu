// backward_differential.cu -- gradients of the differential attention: the kernels of
// backward_kernels.cuh, Delta of both maps, and lambda's gradient carried to its four vectors.
#include "backward_kernels.cuh"

namespace tsa {
namespace {

// Delta of both maps per row, <dO, O1> and <dO, O2> in binary32.  The forward stored O = O1 - lambda O2
// and O2, so the first is <dO, O> + lambda <dO, O2>.  kG = D / 8 threads per row, 16 bytes of each
// tensor per thread, three loads in flight per item and two items per thread.  Rows are laid out per
// map and lane over Sp = nb * 64 tokens; tokens past S get Delta 0 and log-sum-exp +inf.
constexpr int kItems = 2;
template <bool kBF16, int kG>
__global__ void __launch_bounds__(256)
diff_delta(const uint16_t *__restrict__ O, const uint16_t *__restrict__ O2, const uint16_t *__restrict__ dO,
           const float *__restrict__ lse, int S, int Sp, float *__restrict__ delta, float *__restrict__ lse_pad,
           const __grid_constant__ DiffTerms terms, const __grid_constant__ SmallSchedule schedule) {
    if (schedule.nb > 0 && blockIdx.x == gridDim.x - 1) {  // one block more per lane; the first lane's works
        if (blockIdx.y == 0) build_small_schedule(schedule);
        return;
    }
    constexpr int D = kG * 8;
    const long long lane = blockIdx.y;
    const float lam = lambda_of<D / 2, kBF16>(terms, (int)(lane % terms.H));
    const int per_lane = Sp * kG;
    const int first = (int)blockIdx.x * (int)blockDim.x * kItems + (int)threadIdx.x;
    uint4 a[kItems], a2[kItems], g[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const int x = first + k * (int)blockDim.x, t = x / kG;
        a[k] = a2[k] = g[k] = make_uint4(0u, 0u, 0u, 0u);
        if (x < per_lane && t < S) {
            const size_t off = (size_t)(lane * S + t) * D + (size_t)(x % kG) * 8;
            a[k] = __ldg(reinterpret_cast<const uint4 *>(O + off));
            a2[k] = __ldg(reinterpret_cast<const uint4 *>(O2 + off));
            g[k] = __ldg(reinterpret_cast<const uint4 *>(dO + off));
        }
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const int x = first + k * (int)blockDim.x, t = x / kG;
        const uint32_t av[4] = {a[k].x, a[k].y, a[k].z, a[k].w}, bv[4] = {a2[k].x, a2[k].y, a2[k].z, a2[k].w},
                       gv[4] = {g[k].x, g[k].y, g[k].z, g[k].w};
        float s = 0.f, s2 = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float g0 = widen16<kBF16>(gv[q] & 0xFFFFu), g1 = widen16<kBF16>(gv[q] >> 16);
            s = fmaf(widen16<kBF16>(av[q] & 0xFFFFu), g0, s);
            s = fmaf(widen16<kBF16>(av[q] >> 16), g1, s);
            s2 = fmaf(widen16<kBF16>(bv[q] & 0xFFFFu), g0, s2);
            s2 = fmaf(widen16<kBF16>(bv[q] >> 16), g1, s2);
        }
#pragma unroll
        for (int off = kG >> 1; off > 0; off >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, off);
            s2 += __shfl_xor_sync(0xffffffffu, s2, off);
        }
        if (x < per_lane && x % kG == 0) {
            const long long pr = lane * Sp + t, rows = (long long)gridDim.y * S, at = lane * S + t;
            delta[pr] = fmaf(lam, s2, s);
            delta[terms.map_rows + pr] = s2;
            lse_pad[pr] = t < S ? padded_lse(__ldg(lse + at)) : INFINITY;
            lse_pad[terms.map_rows + pr] = t < S ? padded_lse(__ldg(lse + rows + at)) : INFINITY;
        }
    }
}

// lambda's gradient, summed over the lanes of a head (or over all of them) and their tiles in a fixed
// order, and the chain rule to the vectors: lambda = exp(lq1.lk1) - exp(lq2.lk2) + init.  One CTA per
// lambda.  Bound by latency: one float per tile.
template <int kW, bool kBF16>
__global__ void __launch_bounds__(1024)
terms_reduce_lambda(const float *__restrict__ partial, int lanes, int tiles, const __grid_constant__ DiffTerms terms,
                    uint16_t *__restrict__ d_lq1, uint16_t *__restrict__ d_lk1, uint16_t *__restrict__ d_lq2,
                    uint16_t *__restrict__ d_lk2) {
    __shared__ float part[32];
    const int tid = threadIdx.x, head = blockIdx.x;
    // the lanes: head, head + H, .. or all
    const int step = terms.per_head ? terms.H : 1;
    const long long items = (long long)(lanes / step) * tiles;
    float s = 0.f;
    for (long long x = tid; x < items; x += 1024)
        s += partial[(x / tiles * step + (terms.per_head ? head : 0)) * tiles + x % tiles];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((tid & 31) == 0) part[tid >> 5] = s;
    __syncthreads();
    s = part[tid & 31];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    float e1, e2;
    lambda_of<kW, kBF16>(terms, head, &e1, &e2);
    if (tid < kW) {
        const long long at = (long long)head * kW + tid;
        const float up = s * e1, down = -s * e2;
        const uint32_t w1 = pack16x2<kBF16>(up * widen16<kBF16>(terms.lk1[at]), up * widen16<kBF16>(terms.lq1[at]));
        const uint32_t w2 = pack16x2<kBF16>(down * widen16<kBF16>(terms.lk2[at]), down * widen16<kBF16>(terms.lq2[at]));
        d_lq1[at] = (uint16_t)(w1 & 0xFFFFu);
        d_lk1[at] = (uint16_t)(w1 >> 16);
        d_lq2[at] = (uint16_t)(w2 & 0xFFFFu);
        d_lk2[at] = (uint16_t)(w2 >> 16);
    }
}

template <int D, bool kBF16>
tsa_status launch_typed(const BwdLaunch &a, const DiffTerms &terms, const uint16_t *O2, uint16_t *const dlambda[4]) {
    const int Sp = a.nb * kBlock, per_lane = Sp * (D / 8);
    const SmallSchedule g = small_schedule(a);
    const dim3 grid((unsigned)((per_lane + 256 * kItems - 1) / (256 * kItems)) + (g.nb > 0 ? 1u : 0u), (unsigned)a.lanes);
    diff_delta<kBF16, D / 8><<<grid, 256, 0, a.stream>>>(a.O, O2, a.dO, a.lse, a.S, Sp, a.delta, a.lse_pad, terms, g);
    TSA_TRY((launch_grad_kernels<D, kBF16, DiffTerms>(a, terms)));
    terms_reduce_lambda<D / 2, kBF16><<<terms.per_head ? terms.H : 1, 1024, 0, a.stream>>>(
        a.partial, a.lanes, (a.nb + 1) / 2, terms, dlambda[0], dlambda[1], dlambda[2], dlambda[3]);
    return cudaGetLastError() == cudaSuccess ? TSA_OK : TSA_ERR_CUDA;
}

}  // namespace

tsa_status launch_differential_backward(const BwdLaunch &a_in, const DiffTerms &terms, const uint16_t *O2,
                                        uint16_t *const dlambda[4]) {
    BwdLaunch a = a_in;
    TSA_TRY(launch_backward_schedule(&a));
    if (a.D == 64)
        return a.bf16 ? launch_typed<64, true>(a, terms, O2, dlambda) : launch_typed<64, false>(a, terms, O2, dlambda);
    if (a.D == 128)
        return a.bf16 ? launch_typed<128, true>(a, terms, O2, dlambda) : launch_typed<128, false>(a, terms, O2, dlambda);
    return TSA_ERR_UNSUPPORTED;
}

}  // namespace tsa
