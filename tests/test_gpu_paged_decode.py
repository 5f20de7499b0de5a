"""One new token over a paged cache, against the 64-bit form."""
import pytest
import torch

import topology_scheduled_gb300 as tsa
from _cache import attention, close, gathered, page_lists

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _normal(*shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def _lists(rows):
    ptr = [0]
    for r in rows:
        ptr.append(ptr[-1] + len(r))
    return (torch.tensor(ptr, dtype=torch.int32, device=DEV),
            torch.tensor([j for r in rows for j in r] or [0], dtype=torch.int32, device=DEV))


def _case(lengths, H, HK, D, page, dtype, seed=0, fill=float("nan"), most=None):
    """Inputs whose caches hold `fill` in every slot that is no token's."""
    table, pages = page_lists(lengths, page, seed=seed, most=most)
    q = _normal(len(lengths), H, D, dtype=dtype, seed=seed + 1)
    kc, vc = _normal(pages, HK, page, D, dtype=dtype, seed=seed + 2), _normal(pages, HK, page, D, dtype=dtype, seed=seed + 3)
    there = torch.zeros((pages, page), dtype=torch.bool)
    for b, n in enumerate(lengths):
        for k in range(0, n, page):
            there[int(table[b, k // page]), :min(page, n - k)] = True
    for x in (kc, vc):
        x.transpose(1, 2)[~there] = fill
    return q, kc, vc, table


def _check(q, kc, vc, table, lengths, rows=None, block=64, scale=None, **kw):
    lists = (None, None) if rows is None else _lists(rows)
    out = tsa.tsa_paged_attention_decode(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV),
                                         torch.tensor(lengths, dtype=torch.int32, device=DEV), *lists, scale, block=block, **kw)
    assert tsa.tsa_last_device_status() == 0
    for b, n in enumerate(lengths):
        keep = torch.arange(n)
        if rows is not None:
            keep = keep[torch.isin(keep // block, torch.tensor(rows[b], dtype=torch.int64))]
        K, V = (gathered(x, table[b], n)[:, keep] for x in (kc, vc))
        close(out[b], *attention(q[b], K, V, q.shape[1] // kc.shape[1], q.shape[2] ** -0.5 if scale is None else scale,
                                 q.dtype), f"sequence {b} of {n}")
    return out


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,HK", [(1, 1), (4, 4), (6, 2), (8, 1), (9, 1), (16, 1), (17, 1), (40, 2), (32, 4)])
def test_heads_that_share_keys(H, HK, D, dtype):
    lengths = [77, 1, 0, 130, 16]
    _check(*_case(lengths, H, HK, D, 16, dtype), lengths)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_page_sizes_and_lengths(page, D):
    lengths = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 0]
    _check(*_case(lengths, 4, 2, D, page, torch.bfloat16, seed=page), lengths)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("B,H,HK,n", [(1, 16, 16, 1000), (1, 1, 1, 9000), (1, 8, 1, 20000), (1, 3, 3, 4100), (2, 32, 2, 5000),
                                      (40, 8, 8, 600)])
@pytest.mark.parametrize("D", [64, 128])
def test_splits(B, H, HK, n, D, dtype):
    """Lengths that clusters, and parts of clusters, share out."""
    lengths = [max(0, n - 37 * b) for b in range(B)]
    _check(*_case(lengths, H, HK, D, 64, dtype, seed=n), lengths)


@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_schedules(D, page, block):
    lengths = [700, 65, 1, 300, 0, 512]
    g = torch.Generator().manual_seed(block)
    rows = []
    for n in lengths:
        nb = -(-n // block)
        rows.append([j for j in range(nb) if float(torch.rand((), generator=g)) < 0.5])
    rows[2], rows[3] = [0], []      # a row that lists its only block, and one that lists none
    rows[5] = list(range(-(-512 // block)))
    _check(*_case(lengths, 6, 2, D, page, torch.float16, seed=page + block, most=-(-1024 // page)), lengths, rows, block)
    # blocks at or beyond the length hold no keys
    past = [r + [j for j in range(-(-n // block), 1024 // block)] for r, n in zip(rows, lengths)]
    _check(*_case(lengths, 6, 2, D, page, torch.float16, seed=page + block, most=-(-1024 // page)), lengths, past, block)


def test_large_scores_and_scale():
    """Scores whose exponentials would not fit unscaled; one key that takes all; a small scale."""
    lengths = [200, 33]
    q, kc, vc, table = _case(lengths, 4, 2, 64, 32, torch.float16, seed=5)
    _check(q * 20, kc, vc, table, lengths, scale=3.0)
    _check(q, kc, vc, table, lengths, scale=1e-4)


def test_many_small_weights_count():
    """f16: one key of weight 1, and 20000 of 2^-20 each that together make 2 % of the sum."""
    n = 20001
    q, kc, vc, table = _case([n], 1, 1, 64, 64, torch.float16, seed=6)
    q[:] = 0
    q[0, 0, 0] = 1
    kc[..., 0] = 0
    kc[int(table[0, 100]), 0, 3, 0] = 20 * 0.6931472
    vc.nan_to_num_(0)
    kc.nan_to_num_(0)
    vc[..., 5] = 1
    vc[int(table[0, 100]), 0, 3, 5] = 0
    out = _check(q, kc, vc, table, [n], scale=1.0)
    want = 20000 / (20000 + 2.0 ** 20)
    assert abs(float(out[0, 0, 5]) - want) < 0.01 * want


def test_what_is_not_finite():
    """NaN in unused slots reaches nothing (all cases above); a key of -inf score has no weight; a row whose
    every score is -inf is 0; a NaN or +inf score makes its row NaN and no other."""
    lengths = [50, 50, 50, 50]
    q, kc, vc, table = _case(lengths, 2, 2, 64, 16, torch.float16, seed=7)
    q[..., 0] = 1.0
    at = [int(table[b, 1]) for b in range(4)]  # keys 16 .. 31
    kc[at[0], 0, 3, 0] = -float("inf")
    for i in range(4):
        for s in range(16 if i < 3 else 2):
            kc[int(table[1, i]), 1, s, 0] = -float("inf")
    kc[at[2], 1, 0, 7] = float("nan")
    kc[at[3], 0, 15, 0] = float("inf")
    out = tsa.tsa_paged_attention_decode(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV),
                                         torch.tensor(lengths, dtype=torch.int32, device=DEV)).cpu()
    for b in range(4):
        K, V = (gathered(x, table[b], 50) for x in (kc, vc))
        for h in range(2):
            if (b, h) in ((2, 1), (3, 0)):
                assert bool(torch.isnan(out[b, h]).all())
            elif (b, h) == (1, 1):
                assert bool((out[b, h] == 0).all())
            else:
                keep = [k for k in range(50) if (b, h, k) != (0, 0, 19)]
                close(out[b, h:h + 1], *attention(q[b, h:h + 1], K[h:h + 1, keep], V[h:h + 1, keep], 1, 64 ** -0.5, q.dtype),
                      f"{b} {h}")


def test_one_array_of_pages_and_given_buffers():
    lengths = [100, 9]
    q, kc, vc, table = _case(lengths, 4, 2, 128, 32, torch.bfloat16, seed=8, fill=0.0)
    store = torch.full((kc.shape[0], 3, 2, 32, 128), float("nan"), dtype=torch.bfloat16)
    store[:, 0], store[:, 2] = kc, vc
    store = store.to(DEV)
    lens = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    want = tsa.tsa_paged_attention_decode(q.to(DEV), kc.to(DEV), vc.to(DEV), table.to(DEV), lens)
    out = torch.empty_like(want)
    got = tsa.tsa_paged_attention_decode(q.to(DEV), store[:, 0], store[:, 2], table.to(DEV), lens, out=out)
    assert got is out and torch.equal(got, want)
    long = _case([60000], 1, 1, 64, 64, torch.float16, seed=9)
    args = [x.to(DEV) for x in long] + [torch.tensor([60000], dtype=torch.int32, device=DEV)]
    need = tsa.tsa_paged_attention_decode_workspace_bytes(1, 1, 1, 64, 64, long[3].shape[1])
    assert need > 0
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=DEV)
    first = tsa.tsa_paged_attention_decode(*args, workspace=ws[:need])
    assert bool((ws[need:] == 255).all())
    assert torch.equal(first, tsa.tsa_paged_attention_decode(*args))
    with pytest.raises(tsa.TsaError) as e:
        tsa.tsa_paged_attention_decode(*args, workspace=ws[:need - 256])
    assert e.value.status == 5


def test_bad_lists_are_reported_and_left_out():
    lengths = [256, 100]
    q, kc, vc, table = _case(lengths, 2, 1, 64, 64, torch.float16, seed=10, fill=0.0)

    def call(lens, ptr=None, idx=None, tab=table):
        lists = (None, None) if ptr is None else (torch.tensor(ptr, dtype=torch.int32, device=DEV),
                                                  torch.tensor(idx, dtype=torch.int32, device=DEV))
        out = tsa.tsa_paged_attention_decode(q.to(DEV), kc.to(DEV), vc.to(DEV), tab.to(DEV),
                                             torch.tensor(lens, dtype=torch.int32, device=DEV), *lists)
        return tsa.tsa_last_device_status(), out

    status, good = call([256, 100], [0, 2, 4], [0, 3, 0, 1])
    assert status == 0
    none = torch.zeros_like(good[0])
    for lens in ([257, 100], [-1, 100]):
        status, out = call(lens, [0, 2, 4], [0, 3, 0, 1])
        assert status == 8 and torch.equal(out[0], none) and torch.equal(out[1], good[1])
        status, out = call(lens)
        assert status == 8 and torch.equal(out[0], none)
    for ptr in ([0, 2, 5], [0, 2, 1]):
        status, out = call([256, 100], ptr, [0, 3, 0, 1])
        assert status == 8 and torch.equal(out[1], none) and torch.equal(out[0], good[0])
    status, out = call([256, 100], [-1, 2, 4], [0, 3, 0, 1])
    assert status == 8 and torch.equal(out[0], none) and torch.equal(out[1], good[1])
    status, first = call([256, 100], [0, 1, 3], [0, 0, 1])
    assert status == 0
    for idx in ([0, 4, 0, 1], [0, -1, 0, 1], [0, 0, 0, 1]):
        status, out = call([256, 100], [0, 2, 4], idx)  # the second entry is left out
        assert status == 8 and torch.equal(out, first)
    # a page outside the cache leaves its keys out
    for bad in (-1, kc.shape[0], 1 << 30):
        tab = table.clone()
        tab[0, 3] = bad
        status, out = call([256, 100], [0, 2, 4], [0, 3, 0, 1], tab)
        assert status == 8 and torch.equal(out, first)
    tab = table.clone()
    tab[0, 1] = tab[0, 2] = tab[1, 2:] = -7  # of blocks that no row lists
    status, out = call([256, 100], [0, 2, 4], [0, 3, 0, 1], tab)
    assert status == 0 and torch.equal(out, good)
