"""Plain 64-bit forms of the rotary positions and of the paged cache's attention, with element-wise error
bounds; r is the unit roundoff of the inputs' type (2^-8 bf16, 2^-11 f16), eta half its subnormal spacing.

* Rotation.  The reference's angles are exact (rationals, reduced by whole turns) up to binary64.  The kernel's
  fraction of a turn is off by |p| 2^-65 (2^-34 for the largest position: below 2^-31 as an angle), and its lower half,
  2^-32 of a turn, is dropped; the rest of a quarter turn, at most pi / 4, is converted, scaled by a rounded factor and
  rounded: 2.5 2^-24 of it, 1.94 2^-24.  Taylor's series leave out 2^-29 at most and lose 1.1 2^-24 to their roundings;
  the magnitude's own rounding and the product with it lose 2 x 2^-24: a cosine or sine is at most 5.2 2^-24 m off.
  (The bound was derived for 7.2 2^-24 m, sincospif's.)  The two roundings of the pair's sum are 2 x 2^-24 of the
  products: 10 2^-24 m (|a| + |b|) covers all, then the result is rounded (r).
* Attention.  A score is a binary32 sum of D exact products, each step of a tensor core's sum at most 2^-23 off:
  D 2^-23 scale |q|.|k|.  Its scaling and the subtraction of the maximum lose 4 2^-24 (|z| + |max|), exp2 (2 ulp)
  2^-22.  A weight is kept as two numbers: r^2 of it is lost, or in f16 (scaled by 2^14, below that half a
  subnormal step) 2^-39 of the largest.  Binary32 sums of n terms lose n 2^-23 of the magnitudes, the joins of up to 2^10
  parts another 2^10 2^-22.  The denominator has the same errors; the result is rounded (r).
"""
import math
from fractions import Fraction

import torch

U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
ETA = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}

# pi to 60 digits, as a rational
PI = Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59)


def turns(positions, frequencies):
    """cos and sin of positions x frequencies, [n, R / 2], from exact products reduced by whole turns."""
    per = [Fraction(f) / (2 * PI) for f in frequencies]
    angle = torch.tensor([[float(((p * f + Fraction(1, 2)) % 1 - Fraction(1, 2)) * 2 * PI) for f in per]
                          for p in positions], dtype=torch.float64)
    return torch.cos(angle), torch.sin(angle)


def rotated(x, positions, frequencies, interleaved=False, magnitude=1.0, inverse=False):
    """x [.., n, D] rotated, in 64 bits, and the bound before the result's rounding."""
    x = x.detach().cpu().double()
    cos, sin = turns(list(positions), list(frequencies))
    if inverse:
        sin = -sin
    h = cos.shape[1]
    at = (torch.arange(0, 2 * h, 2), torch.arange(1, 2 * h, 2)) if interleaved else (torch.arange(h), torch.arange(h, 2 * h))
    a, b = x[..., at[0]], x[..., at[1]]
    y, bound = x.clone(), torch.zeros_like(x)
    y[..., at[0]] = magnitude * (a * cos - b * sin)
    y[..., at[1]] = magnitude * (b * cos + a * sin)
    e = 10 * 2.0 ** -24 * abs(magnitude) * (a.abs() + b.abs())
    bound[..., at[0]], bound[..., at[1]] = e, e
    return y, bound


def close(got, want, bound, what=""):
    """`got` within `bound` and its own type's rounding of `want`; NaN nowhere."""
    dt = got.dtype
    got = got.detach().cpu().double()
    limit = bound + U[dt] * (want.abs() + bound) + ETA[dt]
    off = (got - want).abs()
    assert bool((off <= limit).all()), (what, float((off - limit).nan_to_num(math.inf).max()), float(off.nan_to_num(math.inf).max()))


def attention(q, K, V, share, scale, dtype):
    """O [H, D] of one sequence's query q [H, D] over its keys K, V [HK, n, D], and the bound."""
    q, K, V = (x.detach().cpu().double() for x in (q, K, V))
    H, D = q.shape
    n = K.shape[1]
    if n == 0:
        return torch.zeros_like(q), torch.zeros_like(q)
    K, V = (x.repeat_interleave(share, 0) for x in (K, V))
    z = scale * torch.einsum("hd,hkd->hk", q, K)
    mag = scale * torch.einsum("hd,hkd->hk", q.abs(), K.abs())
    top = z.max(1, keepdim=True).values
    P = torch.softmax(z, 1)
    u = 2.0 ** -24
    es = 2 * D * u * mag + 4 * u * (z.abs() + top.abs()) + 2.0 ** -22
    small = 2.0 ** -39 if dtype is torch.float16 else 0.0
    lost = U[dtype] ** 2 + 2 * n * u + 2.0 ** -12
    each = P * (es + lost) + small  # of a weight's product with V
    mean = (P * (es + 2 * n * u + 2.0 ** -12)).sum(1, keepdim=True)  # of the denominator
    O = torch.einsum("hk,hkd->hd", P, V)
    # second order: both errors are far below 1
    bound = 1.05 * (torch.einsum("hk,hkd->hd", each, V.abs()) + mean * torch.einsum("hk,hkd->hd", P, V.abs()))
    return O, bound


def page_lists(lengths, page, spare=3, seed=0, most=None):
    """A table of pages in a shuffled order, -1 beyond each sequence's length, and the number of pages."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lengths]
    most = max(1, *need) if most is None else most
    free = torch.randperm(sum(need) + spare, generator=g).tolist()
    table = torch.full((len(lengths), most), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        for i in range(n):
            table[b, i] = free.pop()
    return table, sum(need) + spare


def gathered(cache, table, n):
    """The first n tokens of a sequence whose pages `table` lists: [HK, n, D]."""
    page = cache.shape[2]
    rows = [cache[int(table[k // page]), :, k % page] for k in range(n)]
    return torch.stack(rows, 1) if rows else cache.new_zeros((cache.shape[1], 0, cache.shape[3]))
