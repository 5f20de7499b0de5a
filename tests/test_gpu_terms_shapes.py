"""Single sequences and lanes without a batch: [S, D] and [heads, S, D] give what [1, heads, S, D] gives, forward and
backward."""
import pytest
import torch

import topology_scheduled_gb300 as tsa
from test_gpu_biased import DEV, STARTS, _csr, _dev

pytestmark = pytest.mark.gpu
GEO = STARTS["geometric"]


@pytest.mark.parametrize("which", ["biased", "differential"])
@pytest.mark.parametrize("dims", [2, 3])
def test_shapes(which, dims):
    H, S, D = (1 if dims == 2 else 3), 150, 64
    g = torch.Generator().manual_seed(dims)
    q, k, v, do = (torch.randn((1, H, S, D), generator=g).half().to(DEV) for _ in range(4))
    rp, ci = _dev(*_csr("dense", S, 64))
    if which == "biased":
        extra = ((torch.randn((H, len(GEO)), generator=g)).half().to(DEV), GEO)
        fwd, bwd = tsa.tsa_biased_attention_fwd, tsa.tsa_biased_attention_backward
    else:
        extra = (*((0.2 * torch.randn(D // 2, generator=g)).half().to(DEV) for _ in range(4)), 0.5)
        fwd, bwd = tsa.tsa_differential_attention_fwd, tsa.tsa_differential_attention_backward
    *o, lse = fwd(q, k, v, rp, ci, *extra)
    want = [*o, lse, *bwd(q, k, v, *o, do, lse, rp, ci, *extra)]
    shape = (S, D) if dims == 2 else (H, S, D)
    a, b, c, d = (x.view(shape) for x in (q, k, v, do))
    *o, lse = fwd(a, b, c, rp, ci, *extra)
    got = [*o, lse, *bwd(a, b, c, *o, d, lse, rp, ci, *extra)]
    assert tsa.tsa_last_device_status() == 0
    for x, y in zip(got, want):
        assert x.shape == (shape if y.dim() == 4 else y.shape)
        assert torch.equal(x.reshape(-1), y.reshape(-1))
