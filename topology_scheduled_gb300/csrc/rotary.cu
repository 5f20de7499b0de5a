// rotary.cu -- rotary positions, and new tokens' way into a paged cache (include/tsa_cache.h).
//
// One kernel moves rows of up to three tensors: rotated (Q, K) or as they are (V), to strided rows or to the
// pages of a cache.  Bound by memory: 4 bytes per element, read and written once.
//  * A position's angles are the same for every head, so a thread keeps one token's 8 pairs (two 16-byte
//    vectors of a row) and walks the heads with their cosines and sines in registers.
//  * An angle is a 64-bit fraction of a turn: position times the frequency's fraction, modulo 2^64, which is
//    the reduction by whole turns, exact up to |p| 2^-65 turns at any position, with no binary64 arithmetic.
//    The nearest quarter turn is read off its upper half, and the rest, at most pi / 4, goes through the Taylor
//    series of sine and cosine (to x^9 and x^10; what they leave out is below 2^-29).
//  * A thread's two vectors lie R / 2 dimensions apart in either layout: then each load instruction of a
//    warp covers whole 128-byte lines, and in the half layout the vectors hold the two sides of 8 pairs.
// Measured: [2, 32 + 32 heads, 32768, 128] bf16 from tokens first to heads first (2.1 GB) 310 us = 6.9 TB/s;
// [4, 16 + 16, 8192, 64] f16 43 us = 6.2; 4 x 8192 tokens, 32 + 8 heads, to a cache 116 us; one token 2.8 us.
#include <algorithm>
#include <cmath>

#include "tsa_device.cuh"
#include "tsa_internal.h"

namespace tsa {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;  // heads whose rows a thread has in flight

template <bool kBF16>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
    if constexpr (kBF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}

// Cosine and sine of a fraction of a turn, at most 3 x 2^-24 off: the rounded angle 1.94 (pi / 4 times its conversion,
// factor and product), the series' own roundings and what it leaves out 0.7. (sincospif, measured here: 9 % slower
// on [3,16 heads,1999,128] and on a single token.)
__device__ __forceinline__ void turned(uint64_t phase, float &cs, float &sn) {
    const uint32_t u = (uint32_t)(phase >> 32), quarter = (u + 0x20000000u) >> 30;
    const float x = (float)(int)(u - (quarter << 30)) * (6.283185307179586f * 0x1p-32f), xx = x * x;
    const float s = fmaf(x * xx, fmaf(xx, fmaf(xx, fmaf(xx, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), x);
    const float c = fmaf(xx, fmaf(xx, fmaf(xx, fmaf(xx, fmaf(xx, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f),
                                 -0.5f), 1.f);
    sn = quarter & 1u ? c : s;
    cs = quarter & 1u ? s : c;
    if (quarter & 2u) sn = -sn;
    if ((quarter + 1u) & 2u) cs = -cs;
}

// Elements (a vector's 8, of both vectors) rotated by the pairs' cosines and sines.
template <bool kBF16, bool kInterleaved>
__device__ __forceinline__ void turn(uint4 &lo, uint4 &hi, const float (&cs)[8], const float (&sn)[8]) {
    float x[8], y[8], u[8], v[8];
    widen8<kBF16>(lo, x);
    widen8<kBF16>(hi, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (kInterleaved) {
            // pairs 0..3 in the first vector, 4..7 in the second
            const float *p = i < 4 ? x : y;
            float *o = i < 4 ? u : v;
            const int at = 2 * (i & 3);
            o[at] = fmaf(p[at], cs[i], -p[at + 1] * sn[i]);
            o[at + 1] = fmaf(p[at + 1], cs[i], p[at] * sn[i]);
        } else {
            u[i] = fmaf(x[i], cs[i], -y[i] * sn[i]);
            v[i] = fmaf(y[i], cs[i], x[i] * sn[i]);
        }
    }
    lo = make_uint4(narrow2<kBF16>(u[0], u[1]), narrow2<kBF16>(u[2], u[3]), narrow2<kBF16>(u[4], u[5]),
                    narrow2<kBF16>(u[6], u[7]));
    hi = make_uint4(narrow2<kBF16>(v[0], v[1]), narrow2<kBF16>(v[2], v[3]), narrow2<kBF16>(v[4], v[5]),
                    narrow2<kBF16>(v[6], v[7]));
}

// (The pointers of a part may be the same: rows are read before they are written, by the same thread.)
template <bool kBF16, bool kInterleaved>
__global__ void __launch_bounds__(kThreads)
rows_kernel(const __grid_constant__ RowsLaunch a) {
    wait_for_predecessor();
    const int units = a.D / 16;  // of two 16-byte vectors each, per row
    const int per_cta = kThreads / units;
    const int tid = threadIdx.x;
    const int unit = tid % units;
    const long long n = (long long)blockIdx.x * per_cta + tid / units;  // token of the batch
    if (tid >= per_cta * units || n >= (long long)a.B * a.S) return;
    const int b = (int)(n / a.S), s = (int)(n % a.S);

    int position = s;
    bool there = true;             // the row is a token's
    long long page = -1, slot = 0; // where it goes in the cache
    if (a.seq_lens) {
        const int len = a.seq_lens[b], fresh = a.counts ? a.counts[b] : a.S;
        const bool bad = len < 0 || len > (a.max_pages << a.page_shift) || fresh < 0 || fresh > a.S;
        position = len - fresh + s;
        there = !bad && s < fresh && position >= 0;
        if (bad && s == 0 && unit == 0 && blockIdx.y == 0) raise_status(a.flags, kDevBadSchedule);
        if (there) {
            page = a.page_table[(long long)b * a.max_pages + (position >> a.page_shift)];
            slot = position & ((1 << a.page_shift) - 1);
            if (page < 0 || page >= a.num_pages) {
                if (unit == 0 && blockIdx.y == 0) raise_status(a.flags, kDevBadSchedule);
                page = -1;
            }
        }
    } else if (a.positions) {
        position = a.positions[(a.position_rows > 1 ? (long long)b * a.S : 0) + s];
    }

    // Vectors of the unit: two of the rotated part, R / 2 apart, or two of the copied rest.
    const int turning = a.R / 16;
    const bool turns = unit < turning;
    const int first = turns ? unit : turning + unit;
    const int second = first + (turns ? turning : units - turning);
    float cs[8], sn[8];
    if (turns && there) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int pair = kInterleaved ? 4 * (i < 4 ? first : second) + (i & 3) : 8 * unit + i;
            const unsigned long long phase = (unsigned long long)(long long)position * a.step[pair];
            turned(phase, cs[i], sn[i]);
            sn[i] *= a.magnitude;
            cs[i] *= a.magnitude;
        }
    }

    int at = blockIdx.y * a.heads_per_cta;  // among the parts' heads, one part after the other
    const int end = at + a.heads_per_cta;
    int before = 0;
#pragma unroll
    for (int p = 0; p < 3; ++p) {
        const RowsPart &part = a.part[p];
        const int h0 = max(at - before, 0), h1 = min(end - before, part.heads);
        before += part.heads;
        if (h0 >= h1) continue;
        const bool paged = part.page_stride > 0;
        if (paged && page < 0) continue;
        const uint16_t *from = part.from + b * part.from_batch + s * part.from_token;
        uint16_t *to = part.to + (paged ? page * part.page_stride + slot * a.D : b * part.to_batch + s * part.to_token);
        const int v0 = 8 * (part.rotated ? first : unit), v1 = 8 * (part.rotated ? second : unit + units);
        for (int h = h0; h < h1; h += kUnroll) {
            uint4 lo[kUnroll], hi[kUnroll];
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                if (h + i < h1 && there) {
                    const uint16_t *row = from + (h + i) * part.from_head;
                    lo[i] = *reinterpret_cast<const uint4 *>(row + v0);
                    hi[i] = *reinterpret_cast<const uint4 *>(row + v1);
                } else {
                    lo[i] = hi[i] = make_uint4(0u, 0u, 0u, 0u);
                }
            }
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                if (part.rotated && turns && there) turn<kBF16, kInterleaved>(lo[i], hi[i], cs, sn);
                if (h + i < h1) {
                    uint16_t *row = to + (h + i) * part.to_head;
                    *reinterpret_cast<uint4 *>(row + v0) = lo[i];
                    *reinterpret_cast<uint4 *>(row + v1) = hi[i];
                }
            }
        }
    }
}

}  // namespace

tsa_status launch_rows(RowsLaunch *a, int sms) {
    const int per_cta = kThreads / (a->D / 16);
    const long long tiles = ((long long)a->B * a->S + per_cta - 1) / per_cta;
    int heads = 0;
    for (const RowsPart &p : a->part) heads += p.heads;
    // Heads per thread block: 8, or as many as leave half of the multiprocessors a block.  A block's angles cost
    // as much as two to three heads' rows, but one block's heads are one after the other: us with 1 / 2 / 4 / 8 / 16,
    // [2, 64 heads, 32768, 128] 1098 / 575 / 338 / 310 / 312, [1, 48, 663, 128] 11.6 / 7.8 / 5.3 / 5.2 / 6.7,
    // [3, 16, 1999, 128] 27.6 / 16.1 / 11.0 / 9.2 / 10.7, [1, 32, 1, 64] 3.2 / 3.3 / 3.5 / 4.0 / 5.2 (with sincospif;
    // the series takes 0.3 to 1 us off each).
    int per = 8;
    while (per > 1 && tiles * ((heads + per - 1) / per) < sms / 2) per /= 2;
    a->heads_per_cta = per;
    cudaLaunchAttribute early = set_up_early();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)tiles, (unsigned)((heads + per - 1) / per));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = a->stream;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    void (*kernel)(RowsLaunch) = a->bf16 ? (a->interleaved ? rows_kernel<true, true> : rows_kernel<true, false>)
                                         : (a->interleaved ? rows_kernel<false, true> : rows_kernel<false, false>);
    return launched(cudaLaunchKernelEx(&cfg, kernel, *a));
}

}  // namespace tsa
