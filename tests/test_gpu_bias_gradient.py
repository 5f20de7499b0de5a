"""The gradient of the biases, bucket by bucket, at tolerances far below the values.

The backward call reads the forward's output only for Delta = <dO, O>, and its log-sum-exp.  Here both are
given as the 64-bit form has them: the log-sum-exp rounded to binary32, and an O whose product with dO is Delta
to about 2^-20 of its largest term.  What is left is the error of binary32 scores and sums (see _terms)."""
import pytest
import torch

import topology_scheduled_gb300 as tsa
from _terms import ACC, ETA, U, _close, _weights, allowed, biased, bucket_of, lanes, softmax
from test_gpu_biased import DEV, _csr, _dev

pytestmark = pytest.mark.gpu
D = 64


def _o_for(do, delta):
    """An O of dO's type with <dO, O> = delta: a quotient by dO's largest element of the row, what its rounding
    leaves by the next, and once more.  Returns it with the largest error that is left."""
    O = torch.zeros_like(do)
    rest = delta.clone()
    order = do.abs().argsort(-1, descending=True)
    for i in range(3):
        at = order[..., i:i + 1]
        g = do.gather(-1, at).double().squeeze(-1)
        part = (rest / g).to(do.dtype)
        O.scatter_(-1, at, part.unsqueeze(-1))
        rest = rest - g * part.double()
    return O, rest.abs()


def _run(S, dtype, block, kind, starts, bias, seed, H=1):
    """dbias from the kernel, and its value and bound from the 64-bit form ([H, buckets] each)."""
    g = torch.Generator().manual_seed(seed)
    q, k, v, do = (torch.randn((1, H, S, D), generator=g).to(dtype) for _ in range(4))
    rp, ci = _csr(kind, S, block, seed=1)
    M, at = allowed(rp, ci, S, block), bucket_of(S, starts)
    n, scale = len(starts), D ** -0.5
    value, bound = (torch.zeros((H, n), dtype=torch.float64) for _ in range(2))
    O, lse = torch.zeros_like(do), torch.zeros((H, S), dtype=torch.float32)
    b = bias.double()
    b = torch.where(b <= -1e30, -torch.inf, b)
    for h in range(H):
        qq, kk, vv, gg = (lanes(x)[h] for x in (q, k, v, do))
        P, l64, es = _weights(qq, kk, M, scale, b[h][at], D)
        dP = gg @ vv.T
        delta = (P * dP).sum(-1)
        O[0, h], left = _o_for(do[0, h], delta)
        lse[h] = l64.float()
        dS = P * (dP - delta[:, None])
        # Delta: what is left, and a binary32 sum of three products; dP: one of D; the sums over rows and tiles
        delta_err = left + 3 * ACC * (gg.abs() * O[0, h].double().abs()).sum(-1)
        edP = D * ACC * (gg.abs() @ vv.abs().T)
        err = P * es * (dP - delta[:, None]).abs() + P * (edP + delta_err[:, None]) + 8 * S * ACC * dS.abs()
        last = at == n - 1
        for x in range(n):
            here = at == x
            value[h, x] = dS[here].sum()
            bound[h, x] = err[here].sum()
        rows = (last & M).any(-1)  # the last bucket is minus the sum of the row's others
        bound[h, -1] = err.masked_fill(last, 0)[rows].sum() + (P.sum(-1) - 1).abs().mul(delta.abs())[rows].sum()
    bound = bound + U[dtype] * value.abs() + ETA[dtype]
    args = [x.to(DEV) for x in (q, k, v, O, do, lse)]
    got = tsa.tsa_biased_attention_backward(*args, *_dev(rp, ci), bias.to(DEV), starts, block=block)[3]
    assert tsa.tsa_last_device_status() == 0
    return got, value, bound


@pytest.mark.parametrize("low,dtype", [(-65504.0, torch.float16), (-1e4, torch.float16), (-300.0, torch.bfloat16),
                                       (-1e4, torch.bfloat16), (-3e38, torch.bfloat16)])
@pytest.mark.parametrize("starts", [[0, 1, 8, 70], [0, 40, 300, 301, 400]])
def test_finite_masks_get_no_gradient(low, dtype, starts):
    """Biases so low that no weight of their keys is left, the open last bucket's among them: exactly 0."""
    H, S = 3, 700
    bias = torch.randn((H, len(starts)), generator=torch.Generator().manual_seed(4)).to(dtype)
    bias[0, -1], bias[1, 1], bias[2, -1], bias[2, 2] = low, low, low, low
    got, value, bound = _run(S, dtype, 64, "dense", starts, bias, 5, H)
    _close(got, value, bound, "dbias")
    for h, x in ((0, -1), (1, 1), (2, -1), (2, 2)):
        assert got[h, x] == 0, (h, x, got[h, x])


CASES = {
    # buckets of many distances, within the first 256, beyond them, and beyond the 2048 that are tabulated
    "geometric": (900, torch.float16, 64, "dense", tsa.relative_bucket_starts(32, 128)),
    "wide": (900, torch.bfloat16, 64, "dense", [0, 40, 300, 301, 700]),
    "wide, sparse": (1400, torch.float16, 64, "random", [0, 30, 290, 440, 640, 1000]),
    "coarse blocks": (1400, torch.bfloat16, 128, "random", [0, 64, 256, 512, 1000]),
    "past the table": (2500, torch.float16, 64, "dense", [0, 40, 500, 2100, 2130, 2300]),
    "past the table, geometric": (2600, torch.bfloat16, 64, "dense", tsa.relative_bucket_starts(128, 2400)),
    # more than 32 buckets in the 95 distances of a step
    "every distance from 300": (800, torch.float16, 64, "dense", [0] + list(range(300, 420)) + [600]),
    "every distance from 2100": (2500, torch.bfloat16, 64, "dense", [0] + list(range(2100, 2220)) + [2400]),
    "empty buckets": (2500, torch.float16, 64, "dense", [0, 300, 300, 300, 305, 2050, 2050, 2400, 2450, 2450]),
    "256 buckets": (1000, torch.float16, 64, "dense", list(range(0, 768, 3))),
    "two": (500, torch.bfloat16, 64, "dense", [0, 250]),
    "an unreached last one": (500, torch.float16, 64, "dense", [0, 100, 300, 10 ** 9]),
}


def _whole_numbers(H, S, dtype, seed):
    """Inputs of small whole numbers, so that q.k and dO.v are sums of binary32 without rounding.  dO.v also holds
    waves of the distance, so that a bucket's sum is not a balance of many signs."""
    g = torch.Generator().manual_seed(seed)
    q, k, v, do = (torch.randint(-2, 3, (1, H, S, D), generator=g).double() for _ in range(4))
    t = torch.arange(S).double()
    for i, period in enumerate((97.0, 611.0, 3001.0)):
        for x in (v, do):
            x[..., 2 * i] = torch.round(4 * torch.cos(2 * torch.pi * t / period))
            x[..., 2 * i + 1] = torch.round(4 * torch.sin(2 * torch.pi * t / period))
    return [x.to(dtype) for x in (q, k, v, do)]


def _chains(starts, S, tiles):
    """How many additions in a row a value of each bucket goes through at most: a step's diagonal (32), a
    tile's steps; then the sums by distance of eight warps, or those of a step's 96 distances (7); the warps; the
    tiles, a thirty-second each, and five more.  The last bucket: a row's 32 columns in every step."""
    steps = -(-S // 64)
    n = [32 + steps + 8 * min(max(0, b - a), 256) + 7 + 8 + tiles // 32 + 6 for a, b in zip(starts, starts[1:])]
    return n + [32 * steps + 5 + 8 + tiles // 32 + 6]


def _tight(S, dtype, block, kind, starts, bias, seed, H):
    """As _run, over whole numbers: a score's error is that of its scaling, bias, log-sum-exp and exp2."""
    q, k, v, do = _whole_numbers(H, S, dtype, seed)
    rp, ci = _csr(kind, S, block, seed=1)
    M, at = allowed(rp, ci, S, block), bucket_of(S, starts)
    n, scale = len(starts), D ** -0.5  # a power of two
    value, bound = (torch.zeros((H, n), dtype=torch.float64) for _ in range(2))
    O, lse = torch.zeros_like(do), torch.zeros((H, S), dtype=torch.float32)
    chains = _chains(starts, S, -(-S // 128))
    for h in range(H):
        qq, kk, vv, gg = (lanes(x)[h] for x in (q, k, v, do))
        z = scale * (qq @ kk.T) + bias[h].double()[at]
        P, l64 = softmax(z, M)
        lse[h] = l64.float()
        # in log2 units: the bias, the log-sum-exp and the score are each rounded once or twice, as is their sum
        size = z.abs() + 2 * bias[h].double()[at].abs() + 2 * l64.abs().nan_to_num(0, 0, 0)[:, None]
        es = 4 * ACC * size + 2.0 ** -22  # (exp2: 2 ulp)
        dP = gg @ vv.T
        delta = (P * dP).sum(-1)
        O[0, h], left = _o_for(do[0, h], delta)
        delta_err = left + 3 * ACC * (gg.abs() * O[0, h].double().abs()).sum(-1)
        dS = P * (dP - delta[:, None])
        err = P * (es * (dP - delta[:, None]).abs() + delta_err[:, None]) + 2 * ACC * dS.abs()
        for x in range(n):
            here = at == x
            value[h, x] = dS[here].sum()
            bound[h, x] = (err + chains[x] * ACC * dS.abs())[here].sum()
        last = at == n - 1
        rows = (last & M).any(-1)  # the last bucket is minus the sum of the row's others
        bound[h, -1] = (err + chains[-1] * ACC * dS.abs()).masked_fill(last, 0)[rows].sum()
    bound = bound + U[dtype] * value.abs() + ETA[dtype]
    args = [x.to(DEV) for x in (q, k, v, O, do, lse)]
    got = tsa.tsa_biased_attention_backward(*args, *_dev(rp, ci), bias.to(DEV), starts, block=block)[3]
    assert tsa.tsa_last_device_status() == 0
    return got, value, bound


@pytest.mark.parametrize("case", CASES)
def test_bucket_by_bucket(case):
    S, dtype, block, kind, starts = CASES[case]
    H = 2
    bias = torch.randn((H, len(starts)), generator=torch.Generator().manual_seed(7)).to(dtype)
    got, value, bound = _tight(S, dtype, block, kind, starts, bias, 8, H)
    _close(got, value, bound, "dbias")
    width = torch.tensor([max(0, min(b, S) - a) for a, b in zip(starts, starts[1:] + [S])])
    there = width > 0
    assert bool((value[:, ~there] == 0).all()) and bool((got[:, ~there] == 0).all())
    # The bounds hide no bucket: a sum that is left out, or counted twice, is far over them
    over = value.abs() / bound
    assert bool((over[:, width > 1] > 4).all()) and (over[:, there] > 8).double().mean() > 0.9, over


@pytest.mark.parametrize("width,dtype,block,starts", [(64, torch.float16, 64, [0, 40, 500, 2100, 2130, 2300]),
                                                      (128, torch.bfloat16, 128, tsa.relative_bucket_starts(128, 2400))])
def test_all_gradients_past_the_table(width, dtype, block, starts):
    """dQ, dK and dV where the biases of a step are looked up beyond the 2048 distances that are tabulated."""
    B, H, S = 1, 1, 2500
    g = torch.Generator().manual_seed(width)
    q, k, v, do = (torch.randn((B, H, S, width), generator=g).to(dtype) for _ in range(4))
    bias = (2 * torch.randn((H, len(starts)), generator=g)).to(dtype)
    rp, ci = _csr("dense", S, block)
    ref = biased(q, k, v, rp, ci, block, width ** -0.5, bias, starts, do)
    args = [x.to(DEV) for x in (q, k, v)]
    csr = _dev(rp, ci)
    O, lse = tsa.tsa_biased_attention_fwd(*args, *csr, bias.to(DEV), starts, block=block)
    got = tsa.tsa_biased_attention_backward(*args, O, do.to(DEV), lse, *csr, bias.to(DEV), starts, block=block)
    assert tsa.tsa_last_device_status() == 0
    _close(O, *ref["O"], "O")
    for name, x in zip(("dQ", "dK", "dV", "dbias"), got):
        _close(x, *ref[name], name)
