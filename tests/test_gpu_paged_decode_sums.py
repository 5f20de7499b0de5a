"""The sums of one new token's attention are rounded to the nearest, not down.

Scores are 0, so weights are 1 (2^14 in f16, a scale).  Every warp's first key has a value of 4096, its last step begins with
-4096, and the sixteen or thirty-two keys of each step between add k + 15/16 or k + 7/8 units of 4096's last place to what
the warp holds.  Rounded to the nearest a step loses half a unit, 2^-12, at most; rounded towards 0 it loses those 15/16
(the tensor cores' own sums do that), which over a row adds up to half the answer.
"""
import pytest
import torch

import topology_scheduled_gb300 as tsa
from _cache import U

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("share", [1, 10])
def test_small_values_beside_a_large_one(share, D, dtype):
    B, HK, page, n = 20, 8, 64, 4608  # 160 rows: a thread block of four warps each, whose steps they take in turn
    step = 32 if D == 64 else 16
    small = 1.9375 * 2.0 ** -15
    V = torch.full((n, D), small, dtype=torch.float64)
    V[0:4 * step:step] = 4096
    V[n - 4 * step:n:step] = -4096
    V[:, 1::2] *= -1
    want = (V.sum(0) / n).to(DEV)
    vc = V.to(dtype).to(DEV).reshape(n // page, 1, page, D).expand(-1, HK, -1, -1).contiguous()
    assert torch.equal(vc[:, 0].reshape(n, D).cpu().double(), V)
    kc = torch.randn_like(vc)
    table = torch.arange(n // page, dtype=torch.int32, device=DEV).expand(B, -1).contiguous()
    q = torch.zeros((B, HK * share, D), dtype=dtype, device=DEV)
    out = tsa.tsa_paged_attention_decode(q, kc, vc, table, torch.full((B,), n, dtype=torch.int32, device=DEV))
    assert tsa.tsa_last_device_status() == 0
    # each step half a unit, whichever warp's; the join's and the quotient's roundings are of the small sums
    limit = n / step * 2.0 ** -12 / n + (U[dtype] + 2.0 ** -20) * want.abs() + (2.0 ** -25 if dtype is torch.float16 else 0)
    off = (out.double() - want).abs()
    assert bool((off <= limit).all()), float((off / limit).max())
