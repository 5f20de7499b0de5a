"""One new token with biases of one to 256 buckets, near ones and far ones, against the 64-bit definition."""
import pytest
import torch

import topology_scheduled_gb300 as tsa
from test_gpu_decode import DEV, _inputs, _lists, _reference, _rows
from _terms import _close

pytestmark = pytest.mark.gpu

STARTS = {"one": [0], "two": [0, 1], "every distance": list(range(256)), "far": [0, 40, 300, 301, 2100, 2130, 2500],
          "empty": [0, 0, 0, 700, 700, 2900], "geometric": tsa.relative_bucket_starts(128, 2800),
          "beyond the cache": [0, 10, 10 ** 6, 2 ** 31 - 1], "three apart": list(range(0, 768, 3))}


@pytest.mark.parametrize("starts", STARTS)
@pytest.mark.parametrize("D,dtype,block", [(64, torch.float16, 32), (128, torch.bfloat16, 128)])
def test_buckets(starts, D, dtype, block):
    starts = STARTS[starts]
    B, H, cap = 3, 2, 3001
    lens = [cap, 2, 1234]
    q, k, v = _inputs(B, H, cap, D, dtype, len(starts))
    bias = (2 * torch.randn((H, len(starts)), generator=torch.Generator().manual_seed(3))).to(dtype)
    rows = _rows("some", lens, block, cap, 1)
    want, bound = _reference(q, k, v, lens, rows, block, D ** -0.5, bias, starts)
    out = tsa.tsa_biased_attention_decode(q.to(DEV), k.to(DEV), v.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                                          *_lists(rows), bias.to(DEV), starts, block=block)
    assert tsa.tsa_last_device_status() == 0
    _close(out, want, bound, "O")
