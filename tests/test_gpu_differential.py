"""Differential attention over a schedule, against its 64-bit form."""
import pytest
import torch

import topology_scheduled_gb300 as tsa
from _terms import _close, differential
from test_gpu_biased import DEV, _csr, _dev
from topology_scheduled_gb300.autograd import differential_attention

pytestmark = pytest.mark.gpu
INIT = 0.5


def _inputs(B, H, S, D, dtype, heads, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    q, k, v, do = (torch.randn((B, H, S, D), generator=g).to(dtype) for _ in range(4))
    lam = [(0.2 * torch.randn((heads, D // 2), generator=g)).to(dtype) for _ in range(4)]
    return q * std, k, v, do, lam


CASES = [(1, 1, 1, 64, torch.float16, 64, "dense", 1), (1, 2, 2, 128, torch.bfloat16, 32, "dense", 2),
         (1, 2, 63, 64, torch.bfloat16, 64, "dense", 1), (2, 3, 65, 128, torch.float16, 128, "dense", 3),
         (1, 2, 129, 64, torch.float16, 32, "dense", 2), (2, 2, 384, 64, torch.bfloat16, 64, "holes", 1),
         (1, 2, 640, 128, torch.bfloat16, 64, "random", 2), (1, 3, 1000, 64, torch.float16, 32, "random", 3),
         (1, 2, 1000, 128, torch.float16, 128, "random", 1), (1, 1, 450, 128, torch.bfloat16, 32, "holes", 1),
         (1, 2, 300, 64, torch.float16, 64, "empty", 2), (1, 1, 1500, 64, torch.float16, 64, "diagonal", 1)]


@pytest.mark.parametrize("B,H,S,D,dtype,block,kind,heads", CASES)
def test_forward(B, H, S, D, dtype, block, kind, heads):
    q, k, v, _, lam = _inputs(B, H, S, D, dtype, heads, S + D)
    rp, ci = _csr(kind, S, block, seed=H)
    ref = differential(q, k, v, rp, ci, block, (D / 2) ** -0.5, lam, INIT)
    rows, N = 64, B * H * S  # rows behind the last lane stay as they were
    big, big2 = (torch.full((N + rows, D), 7.0, dtype=dtype, device=DEV) for _ in range(2))
    lse_big = torch.full((2 * N + rows,), 7.0, dtype=torch.float32, device=DEV)
    out, out2 = (x[:N].view(B, H, S, D) for x in (big, big2))
    lse = lse_big[:2 * N].view(2, B * H, S)
    lam_d = [x.to(DEV) for x in lam]
    tsa.tsa_differential_attention_fwd(q.to(DEV), k.to(DEV), v.to(DEV), *_dev(rp, ci), *lam_d, INIT, out=out,
                                       out2=out2, lse=lse, block=block)
    assert tsa.tsa_last_device_status() == 0
    for x in (big[N:], big2[N:], lse_big[2 * N:]):
        assert bool((x == 7.0).all())
    _close(out, *ref["O"], "O")
    _close(out2, *ref["O2"], "O2")
    got, want = lse.cpu().double(), ref["lse"]
    assert torch.equal(torch.isinf(got), torch.isinf(want))
    fin = torch.isfinite(want)
    assert not fin.any() or (got - want)[fin].abs().max() <= 2.0 ** -16  # the log-sum-exp adds exact weights
    # without the backward pass's outputs: the same output
    again = tsa.tsa_differential_attention(q.to(DEV), k.to(DEV), v.to(DEV), *_dev(rp, ci), *lam_d, INIT, block=block)
    assert torch.equal(again, out)


def test_equal_maps_leave_one_minus_lambda():
    """With q1 = q2 and k1 = k2 both maps are the same: O = (1 - lambda) softmax V."""
    B, H, S, D = 1, 2, 500, 128
    q, k, v, _, lam = _inputs(B, H, S, D, torch.float16, 2, 4)
    q[..., 64:], k[..., 64:] = q[..., :64], k[..., :64]
    rp, ci = _csr("random", S, 64, 3)
    ref = differential(q, k, v, rp, ci, 64, 0.125, lam, INIT)
    out = tsa.tsa_differential_attention(q.to(DEV), k.to(DEV), v.to(DEV), *_dev(rp, ci), *(x.to(DEV) for x in lam), INIT)
    _close(out, *ref["O"], "O")
    value = torch.exp((lam[0].double() * lam[1]).sum(1)) - torch.exp((lam[2].double() * lam[3]).sum(1)) + INIT
    plain = tsa.tsa_scheduled_attention(*(torch.cat([x[..., :64], 0 * x[..., 64:]], -1).to(DEV) for x in (q, k)),
                                        v.to(DEV), *_dev(rp, ci), 0.125)
    want = plain.cpu().double() * (1 - value).reshape(1, H, 1, 1)
    _close(out, want, 2.0 ** -9 * (1 + value.abs()).reshape(1, H, 1, 1) * (plain.cpu().double().abs() + 1), "O")


def test_masked_places_may_hold_anything():
    B, H, S, D = 1, 3, 100, 64
    q, k, v, _, lam = _inputs(B, H, S, D, torch.float16, 1, 5)
    rp, ci = _csr("dense", S, 64)
    ref = differential(q[:, :1], k[:, :1], v[:, :1], rp, ci, 64, 32 ** -0.5, lam, INIT)
    k[:, 1], v[:, 1], q[:, 2] = float("nan"), float("inf"), float("nan")
    out = tsa.tsa_differential_attention(q.to(DEV), k.to(DEV), v.to(DEV), *_dev(rp, ci), *(x.to(DEV) for x in lam), INIT)
    assert tsa.tsa_last_device_status() == 0
    _close(out[:, 0], *ref["O"], "O of lane 0")


@pytest.mark.parametrize("block", [32, 64, 128])
def test_bad_rows_are_reported(block):
    S, D = 4 * block, 64
    q, k, v, _, lam = _inputs(1, 1, S, D, torch.float16, 1, 9)
    q, k, v, *lam = (x.to(DEV) for x in (q, k, v, *lam))
    for ptr, idx in (([0, 1, 3, 5, 7], [0, 0, 1, 2, 1, 0, 3]), ([0, 1, 3, 5, 9], [0, 0, 1, 1, 2, 0, 3]),
                     ([-2, 1, 3, 5, 7], [0, 0, 1, 1, 2, 0, 3]), ([0, 1, 3, 5, 7], [0, 0, 1, 1, 3, 0, 3])):
        tsa.tsa_differential_attention(q, k, v, *_dev(ptr, idx), *lam, INIT, block=block)
        assert tsa.tsa_last_device_status() == 8


NAMES = ("dQ", "dK", "dV", "dlq1", "dlk1", "dlq2", "dlk2")
BACKWARD = [(1, 1, 1, 64, torch.float16, 64, "dense", 1), (1, 2, 2, 128, torch.bfloat16, 64, "dense", 2),
            (1, 2, 63, 64, torch.bfloat16, 64, "dense", 1), (3, 2, 65, 128, torch.float16, 128, "dense", 2),
            (2, 2, 384, 64, torch.bfloat16, 64, "holes", 1), (1, 2, 640, 128, torch.bfloat16, 64, "random", 2),
            (1, 3, 1000, 64, torch.float16, 128, "random", 3), (2, 2, 1000, 128, torch.float16, 64, "random", 1),
            (1, 1, 450, 128, torch.bfloat16, 64, "holes", 1), (1, 2, 300, 64, torch.float16, 64, "empty", 2),
            (1, 1, 700, 64, torch.float16, 64, "diagonal", 1)]


@pytest.mark.parametrize("B,H,S,D,dtype,block,kind,heads", BACKWARD)
def test_backward(B, H, S, D, dtype, block, kind, heads):
    q, k, v, do, lam = _inputs(B, H, S, D, dtype, heads, S + D)
    rp, ci = _csr(kind, S, block, seed=H)
    ref = differential(q, k, v, rp, ci, block, (D / 2) ** -0.5, lam, INIT, do)
    rpd, cid = _dev(rp, ci)
    qd, kd, vd, dod, *ld = (x.to(DEV) for x in (q, k, v, do, *lam))
    O, O2, lse = tsa.tsa_differential_attention_fwd(qd, kd, vd, rpd, cid, *ld, INIT, block=block)
    N, rows = B * H * S, 64
    big = [torch.full((N + rows, D), 7.0, dtype=dtype, device=DEV) for _ in range(3)]
    outs = [x[:N].view(B, H, S, D) for x in big]
    got = tsa.tsa_differential_attention_backward(qd, kd, vd, O, O2, dod, lse, rpd, cid, *ld, INIT, block=block,
                                                  dq=outs[0], dk=outs[1], dv=outs[2])
    assert tsa.tsa_last_device_status() == 0
    for x in big:  # rows behind the last lane stay as they were
        assert bool((x[N:] == 7.0).all())
    for name, x in zip(NAMES, got):
        _close(x, *ref[name], name)
    again = tsa.tsa_differential_attention_backward(qd, kd, vd, O, O2, dod, lse, rpd, cid, *ld, INIT, block=block)
    for x, y in zip(got, again):
        assert torch.equal(x, y)


def test_autograd():
    """Vectors of one dimension: one lambda for all heads."""
    B, H, S, D = 2, 2, 200, 64
    q, k, v, do, lam = _inputs(B, H, S, D, torch.float16, 1, 21)
    rp, ci = _csr("random", S, 64, 5)
    ref = differential(q, k, v, rp, ci, 64, 0.2, lam, INIT, do)
    leaves = [x.to(DEV).requires_grad_(True) for x in (q, k, v, *(x[0] for x in lam))]
    differential_attention(*leaves[:3], *_dev(rp, ci), *leaves[3:], INIT, 0.2).backward(do.to(DEV))
    for name, x in zip(NAMES, leaves):
        assert x.grad.shape == x.shape
        _close(x.grad, *ref[name], name)
