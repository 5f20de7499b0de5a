"""Forwards of more than 1024 tiles at D = 64 (differential: three thread blocks per SM): a few of their
heads against the 64-bit forms."""
import pytest
import torch

import topology_scheduled_gb300 as tsa
from _terms import ACC, U, _close, biased, differential
from test_gpu_biased import DEV, STARTS, _csr, _dev

pytestmark = pytest.mark.gpu
INIT = 0.5
STARTS = dict(STARTS, **{"past the table": [0, 40, 2100, 2130, 2300]})  # the kernels tabulate 2048 distances
LOW = torch.finfo(torch.bfloat16).min


def _many(S):
    """Heads that make more than 1024 tiles, of two 64-token blocks even."""
    return 1024 // ((-(-S // 64) + 1) // 2) + 2


def _inputs(H, S, dtype, seed, n):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn((1, H, S, 64), generator=g).to(dtype) for _ in range(3))
    q[:, :, S // 2:] *= 6  # maxima that grow along a row
    bias = (3 * torch.randn((H, n), generator=g)).to(dtype)
    lam = [(0.2 * torch.randn((H, 32), generator=g)).to(dtype) for _ in range(4)]
    return q, k, v, bias, lam


CASES = [(700, torch.float16, 64, "random", "geometric"), (640, torch.bfloat16, 64, "holes", "steps"),
         (1000, torch.float16, 32, "random", "far"), (449, torch.bfloat16, 32, "dense", "fine"),
         (900, torch.bfloat16, 128, "random", "single"), (576, torch.float16, 128, "dense", "empty buckets"),
         (330, torch.float16, 64, "empty", "geometric"), (1500, torch.float16, 64, "diagonal", "fine"),
         (2500, torch.bfloat16, 64, "random", "past the table")]


def _room(q, k, scale, lse):
    """What a row's log-sum-exp may lose to its scores (binary32 sums of 64 exact products, their scaling and
    bias) and to exp2, the sum of its weights and the logarithm."""
    mag = scale * (q.double().abs() @ k.double().abs().T).amax(-1)
    return (64 + 4) * ACC * mag + 8 * ACC * lse.abs().nan_to_num(0, 0, 0) + 2.0 ** -19


def _heads(H):
    return [0, H // 2, H - 1]


@pytest.mark.parametrize("S,dtype,block,kind,starts", CASES)
def test_biased(S, dtype, block, kind, starts):
    starts = STARTS[starts]
    H = _many(S)
    q, k, v, bias, _ = _inputs(H, S, dtype, S, len(starts))
    bias[0, ::3], bias[H - 1, -1] = LOW, -float("inf")
    rp, ci = _csr(kind, S, block, seed=1)
    args = [x.to(DEV) for x in (q, k, v)]
    rpd, cid = _dev(rp, ci)
    rows = 64  # rows behind the last lane stay as they were
    big = torch.full((H * S + rows, 64), 7.0, dtype=dtype, device=DEV)
    out = big[:H * S].view(1, H, S, 64)
    _, lse = tsa.tsa_biased_attention_fwd(*args, rpd, cid, bias.to(DEV), starts, out=out, block=block)
    assert tsa.tsa_last_device_status() == 0
    assert bool((big[H * S:] == 7.0).all())
    for h in _heads(H):
        ref = biased(q[:, h:h + 1], k[:, h:h + 1], v[:, h:h + 1], rp, ci, block, 0.125, bias[h:h + 1], starts)
        _close(out[:, h], *ref["O"], f"O of head {h}")
        got, want = lse[h].cpu().double(), ref["lse"][0]
        assert torch.equal(torch.isinf(got), torch.isinf(want))
        fin = torch.isfinite(want)
        # U: the denominator adds rounded weights
        assert ((got - want).abs() <= U[dtype] + _room(q[0, h], k[0, h], 0.125, want))[fin].all()
    few = tsa.tsa_biased_attention(*(x[:, :2].contiguous() for x in args), rpd, cid, bias[:2].to(DEV), starts, block=block)
    # either is off by the weights' rounding, of at most 4 U of the largest value of V in all
    top = v[:, :2].double().abs().amax().item()
    assert (few.double() - out[:, :2].double()).abs().max() <= 8 * U[dtype] * top


@pytest.mark.parametrize("S,dtype,block,kind,starts", CASES)
def test_differential(S, dtype, block, kind, starts):
    H = _many(S)
    q, k, v, _, lam = _inputs(H, S, dtype, S + 1, 1)
    rp, ci = _csr(kind, S, block, seed=2)
    args = [x.to(DEV) for x in (q, k, v)]
    rpd, cid = _dev(rp, ci)
    lam_d = [x.to(DEV) for x in lam]
    out, out2, lse = tsa.tsa_differential_attention_fwd(*args, rpd, cid, *lam_d, INIT, block=block)
    assert tsa.tsa_last_device_status() == 0
    for h in _heads(H):
        ref = differential(q[:, h:h + 1], k[:, h:h + 1], v[:, h:h + 1], rp, ci, block, 32 ** -0.5, [x[h:h + 1] for x in lam], INIT)
        _close(out[:, h], *ref["O"], f"O of head {h}")
        _close(out2[:, h], *ref["O2"], f"O2 of head {h}")
        got, want = lse[:, h].cpu().double(), ref["lse"][:, 0]
        assert torch.equal(torch.isinf(got), torch.isinf(want))
        fin = torch.isfinite(want)
        room = torch.stack([_room(q[0, h, :, p], k[0, h, :, p], 32 ** -0.5, want[m])
                            for m, p in enumerate((slice(0, 32), slice(32, 64)))])
        assert ((got - want).abs() <= room)[fin].all()
    again = tsa.tsa_differential_attention(*args, rpd, cid, *lam_d, INIT, block=block)
    assert torch.equal(again, out)


def test_wait_that_runs_out_is_reported():
    S, starts = 700, STARTS["geometric"]
    H = _many(S)
    q, k, v, bias, lam = _inputs(H, S, torch.float16, 3, len(starts))
    rp, ci = _dev(*_csr("random", S, 64, seed=1))
    q, k, v, bias, *lam = (x.to(DEV) for x in (q, k, v, bias, *lam))
    for call in (lambda: tsa.tsa_biased_attention(q, k, v, rp, ci, bias, starts),
                 lambda: tsa.tsa_differential_attention(q, k, v, rp, ci, *lam, INIT)):
        want = call()
        assert tsa.tsa_last_device_status() == 0
        tsa.tsa_debug_set_wait_injection(True)
        try:
            call()
            assert tsa.tsa_last_device_status() == 7  # TSA_ERR_TIMEOUT
        finally:
            tsa.tsa_debug_set_wait_injection(False)
        assert torch.equal(call(), want) and tsa.tsa_last_device_status() == 0


def test_bad_rows_are_reported():
    S, H = 256, _many(256)
    starts = STARTS["geometric"]
    q, k, v, bias, _ = (x.to(DEV) if isinstance(x, torch.Tensor) else x for x in _inputs(H, S, torch.float16, 4, len(starts)))
    for ptr, idx in (([0, 1, 3, 5, 7], [0, 0, 1, 2, 1, 0, 3]), ([0, 1, 3, 5, 9], [0, 0, 1, 1, 2, 0, 3]),
                     ([-2, 1, 3, 5, 7], [0, 0, 1, 1, 2, 0, 3]), ([0, 1, 3, 5, 7], [0, 0, 1, 1, 3, 0, 3])):
        tsa.tsa_biased_attention(q, k, v, *_dev(ptr, idx), bias, starts)
        assert tsa.tsa_last_device_status() == 8
