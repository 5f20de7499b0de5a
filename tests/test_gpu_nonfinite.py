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


@pytest.mark.parametrize("which,low", [("plain", -float("inf")), ("biased", -float("inf")), ("plain", -3e38), ("biased", -3e38),
                                       ("differential", -3e38)])  # (a differential form's keys are finite)
@pytest.mark.parametrize("H,S,D,dtype", [(2, 300, 64, torch.float16), (1, 250, 128, torch.bfloat16), (260, 256, 64, torch.bfloat16)])
def test_scores_of_minus_infinity(which, low, H, S, D, dtype):
    """A first block whose scores are all -inf, of infinite keys or by overflow, weighs as one that no row
    lists.  (260 heads: the differential form's layout for many tiles.)"""
    if dtype == torch.float16 and low > -float("inf"):
        low = -65504.0  # (no overflow in f16: weights that are 0 beside any other)
    g = torch.Generator().manual_seed(S)
    q, k, v = (torch.randn((1, H, S, D), generator=g).to(dtype).to(DEV) for _ in range(3))
    q = q.abs() + 0.25
    k[:, :, :64] = low
    bias, lam = _learned(H, D, dtype)
    fwd, _, extra = _calls(which, bias, lam)
    nb = -(-S // 64)
    rows = [list(range(i + 1)) for i in range(nb)]
    got = fwd(q, k, v, *_lists(rows), *extra)
    want = fwd(q, k, v, *_lists([r[1:] for r in rows]), *extra)
    assert tsa.tsa_last_device_status() == 0
    first = 64 if low == -65504.0 else 0  # (rows of that block have no other keys)
    for x, w in zip(got[:-1], want[:-1]):
        assert torch.equal(x[:, :, first:], w[:, :, first:])
    lse, wanted = (x[-1].reshape(-1, H, S) for x in (got, want))
    assert torch.equal(lse[..., first:], wanted[..., first:])
    if not first:
        assert bool((got[0][:, :, :64] == 0).all()) and bool((lse[..., :64] == -float("inf")).all())
