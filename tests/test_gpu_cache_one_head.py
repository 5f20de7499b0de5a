"""A cache of one key head, whose pages are contiguous whatever the stride of that axis."""
import pytest
import torch

import topology_scheduled_gb300 as tsa
from _cache import page_lists

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _normal(*shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_one_key_head_of_any_stride():
    """[pages, page_size, 1, D] transposed: the stride of an axis of one says nothing."""
    lengths, page, D = [70, 9], 32, 64
    table, pages = page_lists(lengths, page, seed=1)
    plain = [_normal(pages, 1, page, D, dtype=torch.float16, seed=i).to(DEV) for i in (1, 2)]
    tokens = [x.reshape(pages, page, 1, D).clone().transpose(1, 2) for x in plain]
    assert tokens[0].stride(1) == D and plain[0].stride(1) == page * D
    q, k = _normal(2, 4, 1, D, dtype=torch.float16, seed=3).to(DEV), _normal(2, 1, 1, D, dtype=torch.float16, seed=4).to(DEV)
    f = tsa.rotary_frequencies(D)
    got = []
    for kc, vc in (plain, tokens):
        out = tsa.tsa_paged_append(q, k, k, kc, vc, table.to(DEV), _ints(lengths), None, f)
        got.append((out, tsa.tsa_paged_attention_decode(out[:, :, 0], kc, vc, table.to(DEV), _ints(lengths)), kc, vc))
    assert tsa.tsa_last_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(*got))
