"""Every step of one new token's attention counts once: rows long enough that a warp looks places up several times, to
the bit.

Scores are 0 or -1000, so weights are 1 or 0 to the last bit; values are small whole numbers that tell groups of 16 keys
apart.  Sums are then whole numbers (below 2^24, or 2^14 times that) without a rounding, in whatever order and however
split, and the answer is their quotient, rounded to 32 bits and then to the outputs' type.
"""
import pytest
import torch

import topology_scheduled_gb300 as tsa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _case(lengths, share, HK, D, page, dtype, seed, cap):
    """Queries that each look at one dimension of the keys, and their answers' parts over all of `cap` keys."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    B, most = len(lengths), cap // page
    hidden = torch.rand((B, HK, cap, share), generator=g, device=DEV) < 0.5
    K = torch.randn((B, HK, cap, D), generator=g, device=DEV, dtype=dtype)
    K[..., :share] = torch.where(hidden, -1000.0, 0.0).to(dtype)
    k = torch.arange(cap, device=DEV)
    of = (k // 16 + 5 * torch.arange(HK, device=DEV)[:, None] + 11 * torch.arange(B, device=DEV)[:, None, None])[..., None]
    V = torch.where(of % D == torch.arange(D, device=DEV), 1 + of // D, 0).to(dtype)
    q = torch.zeros((B, HK, share, D), dtype=dtype, device=DEV)
    q[:, :, torch.arange(share), torch.arange(share)] = 1
    pages = torch.randperm(B * most, generator=g, device=DEV).reshape(B, most)
    kc, vc = (torch.empty((B * most, HK, page, D), dtype=dtype, device=DEV) for _ in range(2))
    for cache, x in ((kc, K), (vc, V)):
        cache[pages.flatten()] = x.reshape(B, HK, most, page, D).transpose(1, 2).flatten(0, 1)
    return q.flatten(1, 2), kc, vc, pages.int(), hidden, V


def _answer(hidden, V, seen, dtype):
    """seen [B, cap]: the keys that count.  Rows all of whose scores are -1000 weigh them evenly."""
    w = (~hidden & seen[:, None, :, None]).double()
    w = torch.where(w.sum(2, keepdim=True) > 0, w, seen[:, None, :, None].double())
    total = w.sum(2)[..., None]
    y = torch.einsum("bhks,bhkd->bhsd", w, V.double())
    return torch.where(total > 0, y.float() / total.float(), 0.0).to(dtype).flatten(1, 2)


def _lengths():
    """A warp looks 2048 keys of its row up at once where the row has one thread block."""
    return [0, 1, 15, 2032, 2047, 2048, 2049, 2064, 2065, 3000, 4079, 4080, 4081, 4095, 4096, 4097, 4113, 4200, 4544, 4543]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D,share,page", [(64, 2, 32), (128, 2, 64), (128, 1, 16), (64, 9, 16), (128, 11, 64)])
def test_long_rows(D, share, page, dtype):
    """160 rows: one thread block each."""
    lengths, HK, cap = _lengths(), 8, 4608
    q, kc, vc, table, hidden, V = _case(lengths, share, HK, D, page, dtype, D + page, cap)
    lens = _ints(lengths)
    out = tsa.tsa_paged_attention_decode(q, kc, vc, table, lens, scale=1.0)
    seen = torch.arange(cap, device=DEV) < lens[:, None]
    assert torch.equal(out, _answer(hidden, V, seen, dtype))
    assert tsa.tsa_last_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D,page,block", [(64, 32, 64), (128, 16, 32), (128, 64, 128), (64, 256, 32)])
def test_long_rows_of_a_schedule(D, page, block, dtype):
    lengths, HK, cap = [n + 1500 if n else 0 for n in _lengths()], 8, 6144
    q, kc, vc, table, hidden, V = _case(lengths, 2, HK, D, page, dtype, D + block, cap)
    g = torch.Generator().manual_seed(block)
    nb = cap // block
    listed = torch.rand((len(lengths), nb), generator=g) < torch.linspace(0.3, 1.0, len(lengths))[:, None]
    listed[4] = False
    rows = [r.nonzero().flatten().tolist() for r in listed]  # blocks past the length among them
    ptr = [0]
    for r in rows:
        ptr.append(ptr[-1] + len(r))
    lens = _ints(lengths)
    out = tsa.tsa_paged_attention_decode(q, kc, vc, table, lens, _ints(ptr), _ints([j for r in rows for j in r]), 1.0, block=block)
    k = torch.arange(cap, device=DEV)
    seen = (k < lens[:, None]) & listed.to(DEV)[:, k // block]
    assert torch.equal(out, _answer(hidden, V, seen, dtype))
    assert tsa.tsa_last_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,HK,n", [(1, 1, 5000), (1, 1, 40000), (1, 4, 40000), (2, 1, 20001), (1, 8, 3000), (20, 2, 3001), (8, 8, 9999)])
def test_split_rows(B, HK, n, D, dtype):
    """Rows that clusters and parts of clusters share out."""
    cap, page = -(-n // 64) * 64, 64
    lengths = [n - 700 * (b % 4) for b in range(B)]
    q, kc, vc, table, hidden, V = _case(lengths, 2, HK, D, page, dtype, n + D, cap)
    lens = _ints(lengths)
    out = tsa.tsa_paged_attention_decode(q, kc, vc, table, lens, scale=1.0)
    seen = torch.arange(cap, device=DEV) < lens[:, None]
    assert torch.equal(out, _answer(hidden, V, seen, dtype))
    assert tsa.tsa_last_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("B,HK,n", [(1, 1, 300), (1, 1, 40000), (20, 8, 4500)])
def test_maxima_that_grow_along_a_row(B, HK, n, dtype):
    """Scores that climb by up to 30 powers of two, so that parts meet with different maxima: each weight is a power of two
    up to exp2's 2^-22, sums lose 2^-23 a step and joins 2^-22 each; 2^-10 of the terms covers rows of 4500 steps and 40 joins."""
    D, page, cap = 64, 64, -(-n // 64) * 64
    q, kc, vc, table, _, _ = _case([n] * B, 1, HK, D, page, dtype, 3, cap)
    g = torch.Generator(device=DEV).manual_seed(5)
    z = (torch.linspace(0, 30, cap, device=DEV).floor() - torch.randint(0, 9, (B, HK, cap), generator=g, device=DEV)).double()
    V = torch.randn((B, HK, cap, D), generator=g, device=DEV).to(dtype)
    q.zero_()
    q[..., 0] = 1
    at = table.long().flatten()
    kc[at, :, :, 0] = z.to(dtype).reshape(B, HK, -1, page).transpose(1, 2).flatten(0, 1)
    vc[at] = V.reshape(B, HK, -1, page, D).transpose(1, 2).flatten(0, 1)
    out = tsa.tsa_paged_attention_decode(q, kc, vc, table, _ints([n] * B), scale=0.6931471805599453)
    w = torch.where(torch.arange(cap, device=DEV) < n, torch.exp2(z - z[..., :n].amax(-1, keepdim=True)), 0.0)
    w = w / w.sum(-1, keepdim=True)
    want, terms = ((w[..., None] * x).sum(2) for x in (V.double(), V.double().abs()))
    eps = torch.finfo(dtype).eps / 2
    assert bool(((out.double() - want).abs() <= 2.0 ** -10 * terms + eps * want.abs()).all())
