"""The weights of one new token's attention keep their bits where values cancel.

Four keys whose values nearly cancel leave the roundings of the weights and of the sums.  With one dimension of the
query not 0 a score is exact before its scaling, and |z| <= 0.7.  In units of 2^-24 of a weight: the scale's and the
product's roundings 1.01 each of |z| and of the maximum, and that of their difference, 3.5 (as a factor, ln 2 of it); in
f16 exponents are taken from 14 below the maximum, whose difference is rounded to 2^-21: 5.5 more; exp2 4 (2^-22); what
the weight's parts leave, 4 in f16 (two of 11 bits), 1 in bf16 (three of 8 bits).  Products of a part and a value are
exact; each of a key's 2 (f16) or 3 (bf16) is a step of a binary32 sum, 2 (2^-23) of the magnitudes at most: 16 or 24.
In all 33 either way; 36 leaves room for second orders.  (A weight of 16 bits is off by 128, one of 11 bits 8192.)
"""
import pytest
import torch

import topology_scheduled_gb300 as tsa
from _cache import ETA, U

pytestmark = pytest.mark.gpu
DEV = "cuda"


def cancelling(B, H, D, dtype, seed):
    """Scores [B, H, 4], values [B, H, 4, D] of `dtype` whose weighted sum nearly cancels; that sum's softmax form in
    64 bits, and its terms' magnitudes."""
    g = torch.Generator().manual_seed(seed)
    z = (torch.rand((B, H, 4), generator=g) * -0.7).to(dtype)
    w = torch.softmax(z.double(), -1)
    v = torch.zeros((B, H, 4, D), dtype=dtype)
    v[:, :, 0] = ((1 + torch.rand((B, H, D), generator=g)) * torch.randint(0, 2, (B, H, D), generator=g).mul(2).sub(1)).to(dtype)
    for k in range(1, 4):  # each takes back what the ones before it leave
        rest = torch.einsum("bhk,bhkd->bhd", w, v.double())
        v[:, :, k] = (-rest / w[:, :, k, None]).to(dtype)
    return z, v, torch.einsum("bhk,bhkd->bhd", w, v.double()), torch.einsum("bhk,bhkd->bhd", w, v.double().abs())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("share", [1, 9])
def test_values_that_cancel(share, D, dtype):
    B, HK, page = 8, 4, 16
    z, v, want, terms = cancelling(B, HK, D, dtype, seed=share + D)
    q = torch.zeros((B, HK, share, D), dtype=dtype)
    q[..., 3] = 1
    kc = torch.zeros((B, HK, page, D), dtype=dtype)
    vc = torch.zeros((B, HK, page, D), dtype=dtype)
    kc[:, :, :4, 3] = z
    vc[:, :, :4] = v
    table = torch.arange(B, dtype=torch.int32)[:, None]
    out = tsa.tsa_paged_attention_decode(q.flatten(1, 2).to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV),
                                         torch.full((B,), 4, dtype=torch.int32, device=DEV), scale=1.0)
    assert tsa.tsa_last_device_status() == 0
    off = (out.cpu().double().reshape(B, HK, share, D) - want[:, :, None]).abs()
    limit = 36 * 2.0 ** -24 * terms + U[dtype] * want.abs() + ETA[dtype]
    assert bool((off <= limit[:, :, None]).all()), float((off / limit[:, :, None]).max())
