"""One lane's rows reach no other lane's results, whatever they hold: a partial last block's tiles end at
their lane's last row, in every attention and its backward."""
import pytest
import torch

import topology_scheduled_gb300 as tsa
from test_gpu_biased import DEV, STARTS, _csr, _dev

pytestmark = pytest.mark.gpu
GEO = STARTS["geometric"]


def _calls(which, H, D, dtype):
    g = torch.Generator().manual_seed(1)
    if which == "plain":
        return tsa.tsa_scheduled_attention_fwd, tsa.tsa_scheduled_attention_backward, ()
    if which == "biased":
        bias = torch.randn((H, len(GEO)), generator=g).to(dtype).to(DEV)
        return tsa.tsa_biased_attention_fwd, tsa.tsa_biased_attention_backward, (bias, GEO)
    lam = [(0.2 * torch.randn((H, D // 2), generator=g)).to(dtype).to(DEV) for _ in range(4)]
    return tsa.tsa_differential_attention_fwd, tsa.tsa_differential_attention_backward, (*lam, 0.5)


def _run(which, tensors, rp, ci, block, grads):
    q, k, v, do = tensors
    fwd, bwd, extra = _calls(which, q.shape[1], q.shape[-1], q.dtype)
    *outs, lse = fwd(q, k, v, rp, ci, *extra, block=block)
    back = bwd(q, k, v, *outs, do, lse, rp, ci, *extra, block=block)[:3] if grads else ()
    assert tsa.tsa_last_device_status() == 0
    return [*(x[0] for x in outs), *(x[0] for x in back), lse.reshape(-1, q.shape[1], q.shape[2]).transpose(0, 1)]


@pytest.mark.parametrize("which", ["plain", "biased", "differential"])
@pytest.mark.parametrize("S,D,dtype,block", [(100, 64, torch.float16, 64), (65, 128, torch.bfloat16, 128),
                                             (1, 64, torch.bfloat16, 64), (97, 128, torch.float16, 32),
                                             (190, 64, torch.bfloat16, 128)])
def test_lanes_apart(which, S, D, dtype, block):
    H = 3
    g = torch.Generator().manual_seed(S)
    clean = [torch.randn((1, H, S, D), generator=g).to(dtype).to(DEV) for _ in range(4)]
    rp, ci = _dev(*_csr("dense", S, block))
    want = _run(which, clean, rp, ci, block, block != 32)
    for bad in (float("nan"), float("inf")):
        for i in range(4):
            dirty = [x.clone() for x in clean]
            dirty[i][:, 1] = bad
            got = _run(which, dirty, rp, ci, block, block != 32)
            for n, (x, y) in enumerate(zip(got, want)):
                for h in (0, 2):
                    assert torch.equal(x[h], y[h]), (bad, i, n, h)
