"""The gradient of the biases, bucket by bucket, at tolerances far below the values.

The backward call reads the forward's output only for Delta = <dO, O>, and its log-sum-exp.  Here both are
given as the 64-bit form has them: the log-sum-exp rounded to binary32, and an O whose product with dO is Delta
to about 2^-20 of its largest term.  What is left is the error of binary32 scores and sums (see _terms)."""
import pytest
import torch

import topology_scheduled_gb300 as tsa
from _terms import ACC, ETA, U, _close, _weights, allowed, bucket_of, lanes
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
