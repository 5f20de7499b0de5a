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


@pytest.mark.parametrize("B,H", [(1, 65535), (65535, 1)])
def test_the_most_lanes(B, H):
    """65535 lanes, the largest grid of every form: the last one is the same as when it runs alone."""
    S, D, dtype = 5, 64, torch.bfloat16
    g = torch.Generator().manual_seed(B)
    q, k, v, do = (torch.randn((B, H, S, D), generator=g).to(dtype).to(DEV) for _ in range(4))
    bias = torch.randn((H, 3), generator=g).to(dtype).to(DEV)
    lam = [(0.2 * torch.randn((H, D // 2), generator=g)).to(dtype).to(DEV) for _ in range(4)]
    rp, ci = _dev(*_csr("dense", S, 64))
    lens = torch.full((B,), S, dtype=torch.int32, device=DEV)
    ptr = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    idx = torch.zeros(B, dtype=torch.int32, device=DEV)

    def run(q, k, v, do, bias, lam, lens, ptr, idx):
        o, lse = tsa.tsa_biased_attention_fwd(q, k, v, rp, ci, bias, [0, 1, 3])
        out = [o, *tsa.tsa_biased_attention_backward(q, k, v, o, do, lse, rp, ci, bias, [0, 1, 3])[:3]]
        o, o2, lse = tsa.tsa_differential_attention_fwd(q, k, v, rp, ci, *lam, 0.5)
        out += [o, o2, *tsa.tsa_differential_attention_backward(q, k, v, o, o2, do, lse, rp, ci, *lam, 0.5)[:3]]
        last = q[:, :, -1].contiguous()
        out += [tsa.tsa_biased_attention_decode(last, k, v, lens, ptr, idx, bias, [0, 1, 3]),
                tsa.tsa_differential_attention_decode(last, k, v, lens, ptr, idx, *lam, 0.5)]
        assert tsa.tsa_last_device_status() == 0
        return [x[-1, -1].clone() for x in out]

    want = run(*(x[-1:, -1:].contiguous() for x in (q, k, v, do)), bias[-1:], [x[-1:] for x in lam], lens[-1:], ptr[:2], idx[:1])
    for x, y in zip(run(q, k, v, do, bias, lam, lens, ptr, idx), want):
        assert torch.equal(x, y)
