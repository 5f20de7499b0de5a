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


def _calls(which, bias, lam):
    if which == "plain":
        return tsa.tsa_scheduled_attention_fwd, tsa.tsa_scheduled_attention_backward, ()
    if which == "biased":
        return tsa.tsa_biased_attention_fwd, tsa.tsa_biased_attention_backward, (bias, GEO)
    return tsa.tsa_differential_attention_fwd, tsa.tsa_differential_attention_backward, (*lam, 0.5)


@pytest.mark.parametrize("which", ["plain", "biased", "differential"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("S,D,dtype", [(130, 64, torch.float16), (200, 128, torch.bfloat16)])
def test_training(which, bad, S, D, dtype):
    """A key of head 1 that is not finite: the rows that see it have no output and no log-sum-exp, and
    no gradient of anything that they touch is a number; rows before it and other heads are as ever."""
    H, t = 3, 70
    g = torch.Generator().manual_seed(S)
    q, k, v, do = (torch.randn((1, H, S, D), generator=g).to(dtype).to(DEV) for _ in range(4))
    q[..., 5] = q[..., D - 5] = 1.0
    bias, lam = _learned(H, D, dtype)
    fwd, bwd, extra = _calls(which, bias, lam)
    rp, ci = tsa.tsa_dense_causal_csr(S, 64)

    def run():
        *o, lse = fwd(q, k, v, rp, ci, *extra)
        grads = bwd(q, k, v, *o, do, lse, rp, ci, *extra)
        assert tsa.tsa_last_device_status() == 0
        return o, lse.reshape(-1, H, S), grads

    o0, lse0, grads0 = run()
    k[0, 1, t, 5] = k[0, 1, t, D - 5] = bad  # of both maps
    o, lse, grads = run()
    others = [0, 2]
    for x, w in zip((*o, *grads[:3]), (*o0, *grads0[:3])):
        assert torch.equal(x[0, others], w[0, others])
    assert torch.equal(lse[:, others], lse0[:, others])
    for x, w in zip(o, o0):
        assert torch.equal(x[0, 1, :t], w[0, 1, :t]) and bool(torch.isnan(x[0, 1, t:]).all())
    assert torch.equal(lse[:, 1, :t], lse0[:, 1, :t]) and bool(torch.isnan(lse[:, 1, t:]).all())
    dq, dk, dv = (x[0, 1] for x in grads[:3])
    assert bool(torch.isnan(dq[t:]).all())
    assert bool(torch.isnan(dk).all()) and bool(torch.isnan(dv).all())  # row S - 1 sees every key
    if which == "biased":
        reached = torch.tensor([s < S for s in GEO], device=DEV)
        assert bool(torch.isnan(grads[3][1, reached]).all()) and torch.equal(grads[3][others], grads0[3][others])
    if which == "differential":
        for x, w in zip(grads[3:], grads0[3:]):
            assert bool(torch.isnan(x[1]).all()) and torch.equal(x[others], w[others])
