"""Parts of one array that share no memory, rotated in place and appended."""
import pytest
import torch

import topology_scheduled_gb300 as tsa
from _cache import close, page_lists, rotated

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _normal(*shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("layout", ["heads first", "each head's together"])
@pytest.mark.parametrize("B,S", [(1, 1), (1, 9), (3, 1), (3, 9)])
def test_parts_of_one_array_in_place(B, S, layout, dtype):
    """Q and K as heads of [B, H + 2 HK, S, D], or beside V in each head's [3, D] of a token, rotated in place and appended."""
    H, D, page = 4, 64, 16
    HK = 2 if layout == "heads first" else H
    f = tsa.rotary_frequencies(D)
    if layout == "heads first":
        x = _normal(B, H + 2 * HK, S, D, dtype=dtype, seed=1)
        parts = lambda y: (y[:, :H], y[:, H:H + HK], y[:, H + HK:])  # noqa: E731
    else:
        x = _normal(B, S, H, 3, D, dtype=dtype, seed=1)
        parts = lambda y: [y[:, :, :, i].transpose(1, 2) for i in range(3)]  # noqa: E731
    whole = x.to(DEV)
    q, k, v = parts(whole)
    tsa.tsa_rotary(q, k, f, out=q, out_k=k)
    for got, part in zip((q, k), parts(x)):
        close(got, *rotated(part, range(S), f))
    assert torch.equal(v.cpu(), parts(x)[2])
    whole = x.to(DEV)
    q, k, v = parts(whole)
    table, pages = page_lists([S] * B, page, seed=2)
    kc, vc = (torch.zeros((pages, HK, page, D), dtype=dtype, device=DEV) for _ in range(2))
    tsa.tsa_paged_append(q, k, v, kc, vc, table.to(DEV), _ints([S] * B), None, f, out=q)
    close(q, *rotated(parts(x)[0], range(S), f))
    assert torch.equal(k.cpu(), parts(x)[1]) and torch.equal(v.cpu(), parts(x)[2])
    for b in range(B):
        for t in range(S):
            assert torch.equal(vc[int(table[b, t // page]), :, t % page], v[b, :, t])
    assert tsa.tsa_last_device_status() == 0
