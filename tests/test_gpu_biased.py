"""Scheduled attention with a relative position bias by buckets, against its 64-bit form."""
import numpy as np
import pytest
import torch

import topology_scheduled_gb300 as tsa
from _terms import U, _close, biased
from test_gpu_backward import _schedule
from topology_scheduled_gb300.autograd import biased_attention
from topology_scheduled_gb300.workloads import random_density_csr

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _inputs(B, H, S, D, dtype, n, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    q, k, v, do = (torch.randn((B, H, S, D), generator=g).to(dtype) for _ in range(4))
    return q * std, k, v, do, torch.randn((H, n), generator=g).to(dtype)


def _csr(kind, S, block, seed=0):
    nb = -(-S // block)
    if kind == "dense":
        return (np.array([i * (i + 1) // 2 for i in range(nb + 1)], np.int32),
                np.array([j for i in range(nb) for j in range(i + 1)], np.int32))
    if kind == "empty":
        return np.zeros(nb + 1, np.int32), np.zeros(0, np.int32)
    return _schedule(kind, nb, seed) if nb > 3 else _csr("dense", S, block)


def _dev(rp, ci):
    return torch.as_tensor(rp, dtype=torch.int32, device=DEV), torch.as_tensor(ci, dtype=torch.int32, device=DEV)


STARTS = {"single": [0], "steps": [0, 1, 2, 3, 4, 6, 9, 14, 21, 33, 64, 100], "far": [0, 40, 300, 301, 1000],
          "geometric": tsa.relative_bucket_starts(32, 128), "fine": list(range(200)), "empty buckets": [0, 0, 5, 5, 5, 90]}
CASES = [(1, 1, 1, 64, torch.float16, 64, "dense", "geometric"), (1, 2, 2, 128, torch.bfloat16, 32, "dense", "steps"),
         (1, 2, 63, 64, torch.bfloat16, 64, "dense", "geometric"), (2, 3, 65, 128, torch.float16, 128, "dense", "single"),
         (1, 2, 129, 64, torch.float16, 32, "dense", "fine"), (2, 2, 384, 64, torch.bfloat16, 64, "holes", "geometric"),
         (1, 2, 640, 128, torch.bfloat16, 64, "random", "far"), (1, 3, 1000, 64, torch.float16, 32, "random", "steps"),
         (1, 2, 1000, 128, torch.float16, 128, "random", "geometric"), (1, 1, 450, 128, torch.bfloat16, 64, "holes", "empty buckets"),
         (1, 2, 300, 64, torch.float16, 64, "empty", "geometric"), (1, 1, 1500, 64, torch.float16, 64, "diagonal", "fine")]


@pytest.mark.parametrize("B,H,S,D,dtype,block,kind,starts", CASES)
def test_forward(B, H, S, D, dtype, block, kind, starts):
    starts = STARTS[starts]
    q, k, v, _, bias = _inputs(B, H, S, D, dtype, len(starts), S + D)
    rp, ci = _csr(kind, S, block, seed=H)
    ref = biased(q, k, v, rp, ci, block, D ** -0.5, bias, starts)
    rows = 64  # rows behind the last lane stay as they were
    big = torch.full((B * H * S + rows, D), 7.0, dtype=dtype, device=DEV)
    lse_big = torch.full((B * H * S + rows,), 7.0, dtype=torch.float32, device=DEV)
    out, lse = big[:B * H * S].view(B, H, S, D), lse_big[:B * H * S].view(B * H, S)
    tsa.tsa_biased_attention_fwd(q.to(DEV), k.to(DEV), v.to(DEV), *_dev(rp, ci), bias.to(DEV), starts, out=out,
                                 lse=lse, block=block)
    assert tsa.tsa_last_device_status() == 0
    assert bool((big[B * H * S:] == 7.0).all()) and bool((lse_big[B * H * S:] == 7.0).all())
    _close(out, *ref["O"], "O")
    got, want = lse.cpu().double(), ref["lse"]
    assert torch.equal(torch.isinf(got), torch.isinf(want))
    fin = torch.isfinite(want)
    assert not fin.any() or (got - want)[fin].abs().max() <= U[dtype] + 2.0 ** -18


@pytest.mark.parametrize("low", [-float("inf"), torch.finfo(torch.bfloat16).min, -1e30])
def test_low_biases_leave_their_keys_out(low):
    """A bucket of -inf or of the type's lowest value has no weight; a row whose keys are all in such
    buckets has none at all."""
    B, H, S, D = 1, 2, 200, 64
    starts = [0, 1, 8, 70]
    q, k, v, _, bias = _inputs(B, H, S, D, torch.bfloat16, 4, 3)
    bias[0, 1], bias[1, 0], bias[1, 3] = low, low, low  # head 1: row 0 sees only itself, and leaves it out
    rp, ci = _csr("dense", S, 64)
    ref = biased(q, k, v, rp, ci, 64, D ** -0.5, bias, starts)
    out, lse = tsa.tsa_biased_attention_fwd(q.to(DEV), k.to(DEV), v.to(DEV), *_dev(rp, ci), bias.to(DEV), starts)
    assert tsa.tsa_last_device_status() == 0
    _close(out, *ref["O"], "O")
    assert bool((out[0, 1, 0] == 0).all()) and lse[1, 0] == -float("inf")


def test_zero_bias_is_the_scheduled_attention():
    """Within both calls' bounds: the bias's steps round a score once more before the exponential."""
    B, H, S, D = 2, 2, 700, 128
    q, k, v, _, bias = _inputs(B, H, S, D, torch.float16, 32, 11)
    rp, ci = random_density_csr(11, 0.4, 2)
    _, bound = biased(q, k, v, rp, ci, 64, D ** -0.5, bias * 0, STARTS["geometric"])["O"]
    q, k, v, bias, rp, ci = (x.to(DEV) for x in (q, k, v, bias, *_dev(rp, ci)))
    got = tsa.tsa_biased_attention(q, k, v, rp, ci, bias * 0, STARTS["geometric"])
    want = tsa.tsa_scheduled_attention(q, k, v, rp, ci)
    _close(got, want.cpu().double().reshape(bound.shape), 2 * bound, "O")


def test_masked_places_may_hold_anything():
    """NaN and infinities in another lane's rows, in blocks that no row lists, and in the keys after
    the query reach no output (V's rows of the diagonal block aside: 0 times infinity)."""
    B, H, S, D = 1, 3, 100, 64
    q, k, v, _, bias = _inputs(B, H, S, D, torch.float16, 32, 5)
    rp, ci = _csr("dense", S, 64)
    ref = biased(q[:, :1], k[:, :1], v[:, :1], rp, ci, 64, 0.125, bias[:1], STARTS["geometric"])
    k[:, 1], v[:, 1], q[:, 2] = float("nan"), float("inf"), float("nan")
    out = tsa.tsa_biased_attention(q.to(DEV), k.to(DEV), v.to(DEV), *_dev(rp, ci), bias.to(DEV), STARTS["geometric"])
    assert tsa.tsa_last_device_status() == 0
    _close(out[:, 0], *ref["O"], "O of lane 0")
    # a block that no row lists
    q, k, v, _, bias = _inputs(1, 1, 192, D, torch.float16, 32, 6)
    rp, ci = np.array([0, 1, 1, 3], np.int32), np.array([0, 0, 2], np.int32)
    ref = biased(q, k, v, rp, ci, 64, 0.125, bias, STARTS["geometric"])
    k[:, :, 64:128], v[:, :, 64:128] = float("nan"), float("inf")
    out = tsa.tsa_biased_attention(q.to(DEV), k.to(DEV), v.to(DEV), *_dev(rp, ci), bias.to(DEV), STARTS["geometric"])
    _close(out, *ref["O"], "O")


def test_bad_rows_are_reported():
    B, H, S, D = 1, 1, 256, 64
    q, k, v, _, bias = (x.to(DEV) for x in _inputs(B, H, S, D, torch.float16, 32, 9))
    for ptr, idx in (([0, 1, 3, 5, 7], [0, 0, 1, 2, 1, 0, 3]),     # a row out of order
                     ([0, 1, 3, 5, 9], [0, 0, 1, 1, 2, 0, 3]),     # a row past the end of col_idx
                     ([-2, 1, 3, 5, 7], [0, 0, 1, 1, 2, 0, 3]),    # a row before its beginning
                     ([0, 1, 3, 5, 7], [0, 0, 1, 1, 3, 0, 3])):    # a block after the row's own
        tsa.tsa_biased_attention(q, k, v, *_dev(ptr, idx), bias, STARTS["geometric"])
        assert tsa.tsa_last_device_status() == 8


BACKWARD = [(1, 1, 1, 64, torch.float16, 64, "dense", "geometric"), (1, 2, 2, 128, torch.bfloat16, 64, "dense", "steps"),
            (1, 2, 63, 64, torch.bfloat16, 64, "dense", "geometric"), (3, 2, 65, 128, torch.float16, 128, "dense", "single"),
            (2, 2, 384, 64, torch.bfloat16, 64, "holes", "geometric"), (1, 2, 640, 128, torch.bfloat16, 64, "random", "far"),
            (1, 3, 1000, 64, torch.float16, 128, "random", "steps"), (2, 2, 1000, 128, torch.float16, 64, "random", "geometric"),
            (1, 1, 450, 128, torch.bfloat16, 64, "holes", "empty buckets"), (1, 2, 300, 64, torch.float16, 64, "empty", "geometric"),
            (1, 1, 700, 64, torch.float16, 64, "diagonal", "fine"), (1, 1, 500, 128, torch.float16, 64, "dense", "fine"),
            (1, 1, 900, 64, torch.bfloat16, 64, "dense", "far")]


@pytest.mark.parametrize("B,H,S,D,dtype,block,kind,starts", BACKWARD)
def test_backward(B, H, S, D, dtype, block, kind, starts):
    starts = STARTS[starts]
    q, k, v, do, bias = _inputs(B, H, S, D, dtype, len(starts), S + D)
    rp, ci = _csr(kind, S, block, seed=H)
    ref = biased(q, k, v, rp, ci, block, D ** -0.5, bias, starts, do)
    rpd, cid = _dev(rp, ci)
    qd, kd, vd, dod, bd = (x.to(DEV) for x in (q, k, v, do, bias))
    O, lse = tsa.tsa_biased_attention_fwd(qd, kd, vd, rpd, cid, bd, starts, block=block)
    N, rows = B * H * S, 64
    big = [torch.full((N + rows, D), 7.0, dtype=dtype, device=DEV) for _ in range(3)]
    outs = [x[:N].view(B, H, S, D) for x in big]
    got = tsa.tsa_biased_attention_backward(qd, kd, vd, O, dod, lse, rpd, cid, bd, starts, block=block, dq=outs[0],
                                            dk=outs[1], dv=outs[2])
    assert tsa.tsa_last_device_status() == 0
    for x in big:  # rows behind the last lane stay as they were
        assert bool((x[N:] == 7.0).all())
    for name, x in zip(("dQ", "dK", "dV", "dbias"), got):
        _close(x, *ref[name], name)
    if starts[-1] >= S:  # a bucket that no distance reaches
        assert bool((got[3][:, -1] == 0).all())
    again = tsa.tsa_biased_attention_backward(qd, kd, vd, O, dod, lse, rpd, cid, bd, starts, block=block)
    for x, y in zip(got, again):
        assert torch.equal(x, y)


def test_backward_with_buckets_left_out():
    """Keys whose bucket is left out get no gradient, nor does the bucket, the open last one included."""
    B, H, S, D = 1, 2, 300, 64
    starts = [0, 1, 8, 70]
    q, k, v, do, bias = _inputs(B, H, S, D, torch.bfloat16, 4, 13)
    bias[0, 3], bias[1, 0], bias[1, 2] = -float("inf"), torch.finfo(torch.bfloat16).min, -1e35
    rp, ci = _csr("dense", S, 64)
    ref = biased(q, k, v, rp, ci, 64, D ** -0.5, bias, starts, do)
    rpd, cid = _dev(rp, ci)
    qd, kd, vd, dod, bd = (x.to(DEV) for x in (q, k, v, do, bias))
    O, lse = tsa.tsa_biased_attention_fwd(qd, kd, vd, rpd, cid, bd, starts)
    got = tsa.tsa_biased_attention_backward(qd, kd, vd, O, dod, lse, rpd, cid, bd, starts)
    assert tsa.tsa_last_device_status() == 0
    for name, x in zip(("dQ", "dK", "dV", "dbias"), got):
        _close(x, *ref[name], name)
    assert got[3][0, 3] == 0 and got[3][1, 0] == 0 and got[3][1, 2] == 0


def test_autograd():
    B, H, S, D = 2, 2, 200, 64
    starts = STARTS["geometric"]
    q, k, v, do, bias = _inputs(B, H, S, D, torch.float16, 32, 21)
    rp, ci = _csr("random", S, 64, 5)
    ref = biased(q, k, v, rp, ci, 64, 0.2, bias, starts, do)
    leaves = [x.to(DEV).requires_grad_(True) for x in (q, k, v, bias)]
    # strided views of the inputs, an expanded upstream gradient
    O = biased_attention(leaves[0].transpose(1, 2).contiguous().transpose(1, 2), *leaves[1:3], *_dev(rp, ci), leaves[3],
                         starts, 0.2)
    O.backward(do.to(DEV))
    for name, x in zip(("dQ", "dK", "dV", "dbias"), leaves):
        _close(x.grad, *ref[name], name)
    leaves = [x.to(DEV).requires_grad_(True) for x in (q, k, v, bias)]
    biased_attention(*leaves[:3], *_dev(rp, ci), leaves[3], starts, 0.2).sum().backward()
    ref = biased(q, k, v, rp, ci, 64, 0.2, bias, starts, torch.ones_like(do))
    for name, x in zip(("dQ", "dK", "dV", "dbias"), leaves):
        _close(x.grad, *ref[name], name)
