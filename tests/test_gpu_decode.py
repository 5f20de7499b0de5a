"""One new token per sequence against a cache, biased and differential, against the 64-bit definition.

Weights stay in binary32 here, so an output is off by its inputs' scores (see _terms), by n 2^-24 of
the sum of magnitudes and by its own rounding."""
import numpy as np
import pytest
import torch

import topology_scheduled_gb300 as tsa
from _terms import ACC, ETA, U, _close

pytestmark = pytest.mark.gpu
DEV = "cuda"
STARTS = tsa.relative_bucket_starts(32, 128)


def _inputs(B, H, cap, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((B, H, D), generator=g).to(dtype)
    k, v = (torch.randn((B, H, cap, D), generator=g).to(dtype) for _ in range(2))
    return q, k, v


def _lists(rows):
    ptr = np.cumsum([0] + [len(r) for r in rows])
    return (torch.tensor(ptr, dtype=torch.int32, device=DEV),
            torch.tensor([j for r in rows for j in r] or [0], dtype=torch.int32, device=DEV))


def _reference(q, k, v, lens, rows, block, scale, bias=None, starts=None, lam=None):
    """(O, bound) [B, H, D]; lam [H, 1, 1]-shaped with its two maps, or None."""
    B, H, D = q.shape
    r, eta = U[q.dtype], ETA[q.dtype]
    q, k, v = q.double(), k.double(), v.double()
    O, bound = torch.zeros_like(q), torch.zeros_like(q)
    for b in range(B):
        keys = [t for j in rows[b] for t in range(j * block, min(lens[b], j * block + block))]
        if not keys:
            continue
        kk, vv = k[b][:, keys], v[b][:, keys]
        w = D if lam is None else D // 2
        for m in range(D // w):
            part = slice(m * w, m * w + w)
            z = scale * torch.einsum("hd,hkd->hk", q[b][:, part], kk[..., part])
            mag = scale * D * torch.einsum("hd,hkd->hk", q[b][:, part].abs(), kk[..., part].abs())
            if bias is not None:
                at = np.searchsorted(starts, lens[b] - 1 - np.array(keys), side="right") - 1
                z = z + bias.double()[:, torch.as_tensor(at)]
            p = torch.nan_to_num(torch.softmax(z, -1))
            es = (mag + 4 * z.abs().nan_to_num(0, 0, 0)) * ACC + 2.0 ** -20
            es = es + (p * es).sum(-1, keepdim=True)
            f = 1.0 if m == 0 else -lam.reshape(H, 1)
            o = torch.einsum("hk,hkd->hd", p, vv)
            O[b] += f * o
            bound[b] += abs(f) * torch.einsum("hk,hkd->hd", p * (2 * es + len(keys) * ACC), vv.abs()) + 2.0 ** -18 * o.abs()
    return O, bound + r * O.abs() + eta


LENS = {"ragged": lambda cap, B: [cap, 0, 1, max(1, cap - 1), cap // 2, min(cap, 63), min(cap, 64)][:B],
        "full": lambda cap, B: [cap] * B}


def _rows(kind, lens, block, cap, seed):
    rng = np.random.default_rng(seed)
    out = []
    for n in lens:
        have = -(-n // block)
        if kind == "all":
            out.append(list(range(have)))
        elif kind == "some":
            out.append(sorted(rng.choice(have, size=max(1, have // 3), replace=False).tolist()) if have else [])
        else:  # every block of the cache, also those behind the length
            out.append(list(range(-(-cap // block))))
    return out


CASES = [(1, 1, 1, 64, torch.float16, 64, "all", "full"), (7, 2, 130, 128, torch.bfloat16, 32, "all", "ragged"),
         (7, 3, 1000, 64, torch.float16, 64, "some", "ragged"), (5, 2, 500, 128, torch.float16, 128, "capacity", "ragged"),
         (1, 2, 6000, 128, torch.bfloat16, 64, "all", "full"), (2, 1, 5001, 64, torch.bfloat16, 128, "some", "full"),
         (40, 33, 100, 64, torch.bfloat16, 32, "all", "full")]


@pytest.mark.parametrize("B,H,cap,D,dtype,block,kind,lens", CASES)
def test_biased(B, H, cap, D, dtype, block, kind, lens):
    lens = LENS[lens](cap, B)
    q, k, v = _inputs(B, H, cap, D, dtype, cap + D)
    bias = torch.randn((H, 32), generator=torch.Generator().manual_seed(1)).to(dtype)
    rows = _rows(kind, lens, block, cap, H)
    want, bound = _reference(q, k, v, lens, rows, block, D ** -0.5, bias, STARTS)
    for b, n in enumerate(lens):  # what lies behind a sequence is not read
        k[b, :, n:], v[b, :, n:] = float("nan"), float("inf")
    big = torch.full((B * H + 4, D), 7.0, dtype=dtype, device=DEV)
    out = big[:B * H].view(B, H, D)
    tsa.tsa_biased_attention_decode(q.to(DEV), k.to(DEV), v.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                                    *_lists(rows), bias.to(DEV), STARTS, out=out, block=block)
    assert tsa.tsa_last_device_status() == 0
    assert bool((big[B * H:] == 7.0).all())
    _close(out, want, bound, "O")


@pytest.mark.parametrize("B,H,cap,D,dtype,block,kind,lens", CASES)
@pytest.mark.parametrize("shared", [False, True])
def test_differential(B, H, cap, D, dtype, block, kind, lens, shared):
    lens = LENS[lens](cap, B)
    q, k, v = _inputs(B, H, cap, D, dtype, cap + D + 1)
    g = torch.Generator().manual_seed(2)
    vec = [(0.2 * torch.randn((1 if shared else H, D // 2), generator=g)).to(dtype) for _ in range(4)]
    lam = (torch.exp((vec[0].double() * vec[1]).sum(1)) - torch.exp((vec[2].double() * vec[3]).sum(1)) + 0.4).expand(H)
    rows = _rows(kind, lens, block, cap, H)
    want, bound = _reference(q, k, v, lens, rows, block, (D / 2) ** -0.5, lam=lam)
    for b, n in enumerate(lens):
        k[b, :, n:], v[b, :, n:] = float("nan"), float("inf")
    out = tsa.tsa_differential_attention_decode(q.to(DEV), k.to(DEV), v.to(DEV),
                                                torch.tensor(lens, dtype=torch.int32, device=DEV), *_lists(rows),
                                                *(x.to(DEV) for x in vec), 0.4, block=block)
    assert tsa.tsa_last_device_status() == 0
    _close(out, want, bound, "O")


def test_buckets_left_out():
    B, H, cap, D = 2, 2, 300, 64
    q, k, v = _inputs(B, H, cap, D, torch.bfloat16, 4)
    starts = [0, 1, 8, 70]
    bias = torch.randn((H, 4), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    bias[0, 3], bias[1, 0], bias[1, 1] = -float("inf"), torch.finfo(torch.bfloat16).min, -1e30
    lens, rows = [300, 8], [[0, 1, 2, 3, 4], [0]]  # head 1 of sequence 1 sees only what is left out
    want, bound = _reference(q, k, v, lens, rows, 64, D ** -0.5, torch.where(bias <= -1e30, -float("inf"), bias), starts)
    out = tsa.tsa_biased_attention_decode(q.to(DEV), k.to(DEV), v.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                                          *_lists(rows), bias.to(DEV), starts)
    assert tsa.tsa_last_device_status() == 0
    _close(out, want, bound, "O")
    assert bool((out[1, 1] == 0).all())


def test_agrees_with_the_prompt_form():
    """The last row of the forward over a prompt is the decode of its last token, within both bounds:
    the forward rounds its weights."""
    B, H, S, D = 2, 3, 333, 128
    q, k, v = (x.to(DEV) for x in _inputs(B, H, S, D, torch.float16, 8))
    g = torch.Generator().manual_seed(5)
    Q = torch.randn((B, H, S, D), generator=g).to(torch.float16).to(DEV)
    bias = torch.randn((H, 32), generator=g).to(torch.float16).to(DEV)
    rp, ci = tsa.tsa_dense_causal_csr(S, 64)
    full = tsa.tsa_biased_attention(Q, k, v, rp, ci, bias, STARTS)[:, :, -1]
    lens = torch.full((B,), S, dtype=torch.int32, device=DEV)
    rows = [list(range(6))] * B
    one = tsa.tsa_biased_attention_decode(Q[:, :, -1].contiguous(), k, v, lens, *_lists(rows), bias, STARTS)
    want, bound = _reference(Q[:, :, -1].cpu(), k.cpu(), v.cpu(), [S] * B, rows, 64, D ** -0.5, bias.cpu(), STARTS)
    _close(one, want, bound, "decode")
    top = v.cpu().double().abs().amax(2)
    _close(full, want, bound + 2 * U[torch.float16] * top, "forward")


def test_bad_rows_are_reported():
    B, H, cap, D = 2, 1, 256, 64
    q, k, v = (x.to(DEV) for x in _inputs(B, H, cap, D, torch.float16, 9))
    bias = torch.zeros((H, 32), dtype=torch.float16, device=DEV)

    def status(lens, ptr, idx):
        tsa.tsa_biased_attention_decode(q, k, v, torch.tensor(lens, dtype=torch.int32, device=DEV),
                                        torch.tensor(ptr, dtype=torch.int32, device=DEV),
                                        torch.tensor(idx, dtype=torch.int32, device=DEV), bias, STARTS)
        return tsa.tsa_last_device_status()

    assert status([256, 100], [0, 2, 4], [0, 3, 0, 1]) == 0
    assert status([257, 100], [0, 2, 4], [0, 3, 0, 1]) == 8   # longer than the cache
    assert status([-1, 100], [0, 2, 4], [0, 3, 0, 1]) == 8
    assert status([256, 100], [0, 2, 5], [0, 3, 0, 1]) == 8   # past the end of col_idx
    assert status([256, 100], [-1, 2, 4], [0, 3, 0, 1]) == 8
    assert status([256, 100], [0, 2, 4], [0, 4, 0, 1]) == 8   # a block outside the cache
    assert status([256, 100], [0, 2, 4], [0, -1, 0, 1]) == 8
    assert status([256, 100], [0, 2, 4], [1, 0, 0, 1]) == 8   # out of order
    assert status([256, 100], [0, 2, 4], [1, 1, 0, 1]) == 8   # the same block twice
