// backward_biased.cu -- gradients of the scheduled attention with a bias by buckets: the kernels of
// backward_kernels.cuh, and the sum of the tiles' parts of the bias's gradient.
#include "backward_kernels.cuh"

namespace tsa {
namespace {

// dbias[h][b] = sum over the batch and the tiles, always in the same order, rounded to the inputs'
// type once.  One CTA per head and 32 buckets: a lane per bucket, a warp per slice of the tiles (rows
// of n floats, so a warp reads 128 consecutive bytes), the slices joined through shared memory.
// Bound by latency: at [1, 32, 32768, 128] the parts are 0.5 MB.
constexpr int kReduceWarps = 32;
template <bool kBF16>
__global__ void __launch_bounds__(kReduceWarps * 32)
terms_reduce_bias(const float *__restrict__ partial, int lanes, int H, int tiles, int n, uint16_t *__restrict__ dbias) {
    __shared__ float part[kReduceWarps][33];
    const int h = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.y * 32 + lane;
    const int rows = lanes / H * tiles;
    float s = 0.f;
    if (b < n)
        for (int r = warp; r < rows; r += kReduceWarps)
            s += partial[((long long)(r / tiles * H + h) * tiles + r % tiles) * n + b];
    part[warp][lane] = s;
    __syncthreads();
    // warp w joins bucket w's slices
    s = part[lane][warp];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int to = blockIdx.y * 32 + warp;
    if (lane == 0 && to < n) dbias[(long long)h * n + to] = (uint16_t)(pack16x2<kBF16>(s, 0.f) & 0xFFFFu);
}

}  // namespace

tsa_status launch_biased_backward(const BwdLaunch &a_in, const BiasTerms &terms, uint16_t *dbias) {
    BwdLaunch a = a_in;
    TSA_TRY(launch_backward_schedule(&a));
    TSA_TRY(launch_backward_delta(a));
    TSA_TRY(launch_gradients(a, terms));
    const dim3 grid((unsigned)terms.H, (unsigned)((terms.n + 31) / 32));
    const int tiles = (a.nb + 1) / 2;
    if (a.bf16)
        terms_reduce_bias<true><<<grid, kReduceWarps * 32, 0, a.stream>>>(a.partial, a.lanes, terms.H, tiles, terms.n, dbias);
    else
        terms_reduce_bias<false><<<grid, kReduceWarps * 32, 0, a.stream>>>(a.partial, a.lanes, terms.H, tiles, terms.n, dbias);
    return cudaGetLastError() == cudaSuccess ? TSA_OK : TSA_ERR_CUDA;
}

}  // namespace tsa
