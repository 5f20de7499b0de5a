"""Keys that are not finite, in places that count: what the definition makes NaN is NaN, and nothing else."""
import pytest
import torch

import topology_scheduled_gb300 as tsa
from test_gpu_biased import DEV, STARTS
from test_gpu_decode import _inputs as _cache, _lists

pytestmark = pytest.mark.gpu
GEO = STARTS["geometric"]


def _learned(H, D, dtype):
    g = torch.Generator().manual_seed(2)
    return (torch.randn((H, len(GEO)), generator=g).to(dtype).to(DEV),
            [(0.2 * torch.randn((H, D // 2), generator=g)).to(dtype).to(DEV) for _ in range(4)])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", [0, 63])  # the column: of either map's half
@pytest.mark.parametrize("D,dtype", [(64, torch.float16), (128, torch.bfloat16)])
def test_decode(bad, where, D, dtype):
    """A NaN score, or an infinite one, leaves no weight that is a number; other heads do not see it."""
    B, H, cap = 2, 3, 700
    q, k, v = (x.to(DEV) for x in _cache(B, H, cap, D, dtype, 3))
    q[:, :, where] = 1.0  # an infinity of the key becomes a score of +inf
    bias, lam = _learned(H, D, dtype)
    lens = torch.tensor([cap, 200], dtype=torch.int32, device=DEV)
    lists = _lists([list(range(11)), list(range(4))])

    def both():
        out = (tsa.tsa_biased_attention_decode(q, k, v, lens, *lists, bias, GEO),
               tsa.tsa_differential_attention_decode(q, k, v, lens, *lists, *lam, 0.5))
        assert tsa.tsa_last_device_status() == 0
        return out

    want = both()
    k[0, 1, 555, where] = bad
    k[1, 2, 7, where] = bad
    for x, w in zip(both(), want):
        hit = torch.zeros((B, H), dtype=torch.bool, device=DEV)
        hit[0, 1] = hit[1, 2] = True
        assert bool(torch.isnan(x[hit]).all())
        assert torch.equal(x[~hit], w[~hit])
