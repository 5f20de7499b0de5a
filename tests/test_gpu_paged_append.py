"""New tokens to a paged cache: every slot of the caches and every row of the rotated queries, against the
64-bit form and against tsa_rotary bit for bit."""
import pytest
import torch

import topology_scheduled_gb300 as tsa
from _cache import close, page_lists, rotated

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _normal(*shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def _case(B, H, HK, T, D, page, lengths, dtype, seed=0, most=None):
    table, pages = page_lists([max(0, n) for n in lengths], page, seed=seed, most=most)
    return dict(q=_normal(B, H, T, D, dtype=dtype, seed=seed + 1), k=_normal(B, HK, T, D, dtype=dtype, seed=seed + 2),
                v=_normal(B, HK, T, D, dtype=dtype, seed=seed + 3), kc=_normal(pages, HK, page, D, dtype=dtype, seed=seed + 4),
                vc=_normal(pages, HK, page, D, dtype=dtype, seed=seed + 5), table=table)


def _expected(c, lengths, counts, f, interleaved, magnitude):
    """Caches and queries as they must be after the call; a bound for each."""
    B, T, page = c["q"].shape[0], c["q"].shape[2], c["kc"].shape[2]
    kc, vc, q = c["kc"].double(), c["vc"].double(), torch.zeros(c["q"].shape, dtype=torch.float64)
    ek, eq = torch.zeros_like(kc), torch.zeros_like(q)
    for b in range(B):
        for t in range(counts[b]):
            p = lengths[b] - counts[b] + t
            if p < 0:
                continue
            at, slot = int(c["table"][b, p // page]), p % page
            vc[at, :, slot] = c["v"][b, :, t].double()
            if f is None:
                kc[at, :, slot] = c["k"][b, :, t].double()
                continue
            y, e = rotated(c["k"][b, :, t:t + 1], [p], f, interleaved, magnitude)
            kc[at, :, slot], ek[at, :, slot] = y[:, 0], e[:, 0]
            y, e = rotated(c["q"][b, :, t:t + 1], [p], f, interleaved, magnitude)
            q[b, :, t], eq[b, :, t] = y[:, 0], e[:, 0]
    return kc, ek, vc, q, eq


SHAPES = [  # B, H, HK, T, D, page, lengths after, counts (None: T each)
    (1, 1, 1, 1, 64, 16, [1], None),
    (1, 16, 16, 1, 64, 16, [1000], None),
    (5, 8, 2, 1, 128, 64, [17, 64, 65, 0, 1], None),            # idle: length 0
    (3, 4, 1, 40, 64, 32, [40, 100, 71], None),
    (3, 4, 4, 40, 128, 16, [40, 7, 0], None),                   # padded in front
    (4, 6, 3, 33, 64, 128, [33, 150, 20, 90], [33, 0, 7, 32]),  # padded behind
    (2, 3, 1, 20, 128, 256, [5, 300], [12, 20]),                # longer counts than the sequence
    (70, 2, 1, 1, 64, 16, list(range(70)), None),
]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_against_the_definition(shape, interleaved, dtype):
    B, H, HK, T, D, page, lengths, counts = shape
    c = _case(B, H, HK, T, D, page, lengths, dtype)
    f = tsa.rotary_frequencies(D // 2, 500.0)
    kc, vc = c["kc"].to(DEV), c["vc"].to(DEV)
    n = None if counts is None else torch.tensor(counts, dtype=torch.int32, device=DEV)
    out = tsa.tsa_paged_append(c["q"].to(DEV), c["k"].to(DEV), c["v"].to(DEV), kc, vc, c["table"].to(DEV),
                               torch.tensor(lengths, dtype=torch.int32, device=DEV), n, f, interleaved=interleaved,
                               magnitude=0.75)
    assert tsa.tsa_last_device_status() == 0
    wk, ek, wv, wq, eq = _expected(c, lengths, counts or [T] * B, f, interleaved, 0.75)
    close(kc, wk, ek, "K")
    assert torch.equal(vc.cpu().double(), wv)
    close(out, wq, eq, "Q")
    untouched = ek.amax(-1) == 0  # whole slots as they were, bit for bit
    assert torch.equal(kc.cpu()[untouched], c["kc"][untouched])
    for b in range(B):
        for t in range(T):
            if t >= (counts or [T] * B)[b] or lengths[b] - (counts or [T] * B)[b] + t < 0:
                assert bool((out[b, :, t] == 0).all())


def test_as_it_is():
    """Without frequencies keys go in as they are, NaN and infinities too."""
    lengths = [20, 3]
    c = _case(2, 1, 2, 5, 64, 16, lengths, torch.bfloat16)
    c["k"][0, 1, 2, 3], c["v"][1, 0, 4, 60] = float("nan"), float("inf")
    kc, vc = c["kc"].to(DEV), c["vc"].to(DEV)
    got = tsa.tsa_paged_append(None, c["k"].to(DEV), c["v"].to(DEV), kc, vc, c["table"].to(DEV),
                               torch.tensor(lengths, dtype=torch.int32, device=DEV))
    assert got is None and tsa.tsa_last_device_status() == 0
    wk, _, wv, _, _ = _expected(c, lengths, [5, 5], None, False, 1.0)
    assert torch.equal(kc.cpu().double().nan_to_num(12345.0), wk.nan_to_num(12345.0))
    assert torch.equal(vc.cpu().double(), wv)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_views_and_one_array_of_pages(dtype):
    """Heads of a joint projection, Q in place; keys and values of a page side by side in one array of layers."""
    B, T, H, HK, D, page = 2, 9, 4, 2, 64, 16
    lengths = [9, 30]
    c = _case(B, H, HK, T, D, page, lengths, dtype, seed=7)
    joint = torch.cat([c["q"], c["k"], c["v"]], 1).transpose(1, 2).contiguous().to(DEV)  # [B, T, heads, D]
    q, k, v = (joint[:, :, i:j].transpose(1, 2) for i, j in ((0, H), (H, H + HK), (H + HK, H + 2 * HK)))
    pages = c["kc"].shape[0]
    store = torch.full((3, pages, 2, HK, page, D), 5.0, dtype=dtype, device=DEV)
    store[1, :, 0], store[1, :, 1] = c["kc"].to(DEV), c["vc"].to(DEV)
    kc, vc = store[1, :, 0], store[1, :, 1]
    f = tsa.rotary_frequencies(D)
    lens = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    out = tsa.tsa_paged_append(q, k, v, kc, vc, c["table"].to(DEV), lens, None, f, out=q)
    assert tsa.tsa_last_device_status() == 0 and out.data_ptr() == joint.data_ptr()
    wk, ek, wv, wq, eq = _expected(c, lengths, [T] * B, f, False, 1.0)
    close(kc, wk, ek, "K")
    assert torch.equal(vc.cpu().double(), wv)
    close(q, wq, eq, "Q")
    assert torch.equal(k.cpu(), c["k"]) and torch.equal(v.cpu(), c["v"])
    assert bool((store[0] == 5).all()) and bool((store[2] == 5).all())
    # one key head for all of a projection's, and the rotation of tsa_rotary, bit for bit
    kc2, vc2 = c["kc"].to(DEV), c["vc"].to(DEV)
    one = c["k"][:, :1].to(DEV)
    tsa.tsa_paged_append(None, one.expand(B, HK, T, D), one.expand(B, HK, T, D), kc2, vc2, c["table"].to(DEV), lens, None, f)
    for b in range(B):
        pos = torch.arange(lengths[b] - T, lengths[b], dtype=torch.int32, device=DEV)
        want = tsa.tsa_rotary(one[b:b + 1], None, f, pos)[0, 0]
        for t in range(T):
            p = int(pos[t])
            at = int(c["table"][b, p // page])
            for h in range(HK):
                assert torch.equal(kc2[at, h, p % page], want[t]) and torch.equal(vc2[at, h, p % page], one[b, 0, t])


def test_bad_lists_are_reported_and_left_out():
    B, T, page, D = 3, 2, 16, 64
    c = _case(B, 1, 1, T, D, page, [20, 20, 20], torch.float16)
    f = tsa.rotary_frequencies(D)

    def call(lengths, counts, table):
        kc, vc = c["kc"].to(DEV), c["vc"].to(DEV)
        out = tsa.tsa_paged_append(c["q"].to(DEV), c["k"].to(DEV), c["v"].to(DEV), kc, vc, table.to(DEV),
                                   torch.tensor(lengths, dtype=torch.int32, device=DEV),
                                   None if counts is None else torch.tensor(counts, dtype=torch.int32, device=DEV), f)
        return out, kc, vc, tsa.tsa_last_device_status()

    good = call([20, 20, 20], None, c["table"])
    assert good[3] == 0
    for lengths, counts in (([20, 33, 20], None), ([20, -1, 20], None), ([20, 20, 20], [2, 3, 2]), ([20, 20, 20], [2, -1, 2])):
        out, kc, vc, status = call(lengths, counts, c["table"])
        assert status == 8
        # sequence 1 has no tokens; the others are as they were
        assert bool((out[1] == 0).all()) and torch.equal(out[[0, 2]], good[0][[0, 2]])
        mine = int(c["table"][1, 1])
        assert torch.equal(kc[mine].cpu(), c["kc"][mine]) and torch.equal(vc[mine].cpu(), c["vc"][mine])
        rest = [i for i in range(kc.shape[0]) if i != mine]
        assert torch.equal(kc[rest], good[1][rest]) and torch.equal(vc[rest], good[2][rest])
    for bad in (-1, c["kc"].shape[0], 1 << 30):
        table = c["table"].clone()
        table[1, 1] = bad
        out, kc, vc, status = call([20, 20, 20], None, table)
        assert status == 8 and torch.equal(out, good[0])  # the queries have positions all the same
        mine = int(c["table"][1, 1])
        assert torch.equal(kc[mine].cpu(), c["kc"][mine])
    # an entry that no token reaches may hold anything
    table = c["table"].clone()
    table[:, 0] = -5
    assert call([20, 20, 20], None, table)[3] == 0
