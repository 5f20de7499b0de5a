"""The autograd wrappers with inputs and upstream gradients that are slices of other tensors, at elements that
no 16-byte boundary meets: the same results as for copies of them."""
import pytest
import torch

import topology_scheduled_gb300 as tsa
from test_gpu_biased import DEV, STARTS, _csr, _dev
from topology_scheduled_gb300.autograd import biased_attention, differential_attention, scheduled_attention

pytestmark = pytest.mark.gpu
GEO = STARTS["geometric"]


def _sliced(x, at):
    """A contiguous view of `x`'s values that starts `at` elements into a longer tensor."""
    flat = torch.cat([torch.zeros(at, dtype=x.dtype, device=DEV), x.reshape(-1).to(DEV)])
    return flat[at:].view(x.shape)


@pytest.mark.parametrize("which", ["plain", "biased", "differential"])
@pytest.mark.parametrize("at", [1, 3, 8])
def test_slices(which, at):
    B, H, S, D = 1, 2, 150, 64
    g = torch.Generator().manual_seed(at)
    q, k, v, do = (torch.randn((B, H, S, D), generator=g).half() for _ in range(4))
    learned = {"plain": [], "biased": [torch.randn((H, len(GEO)), generator=g).half()],
               "differential": [(0.2 * torch.randn((H, D // 2), generator=g)).half() for _ in range(4)]}[which]
    rp, ci = _dev(*_csr("dense", S, 64))

    def step(place, joined):
        leaves = [place(x).detach().requires_grad_(True) for x in (q, k, v, *learned)]
        if which == "plain":
            y = scheduled_attention(*leaves, rp, ci)
        elif which == "biased":
            y = biased_attention(*leaves[:3], rp, ci, leaves[3], GEO)
        else:
            y = differential_attention(*leaves[:3], rp, ci, *leaves[3:], 0.5)
        up = do.to(DEV)
        if joined:  # the gradient of y is then a slice, from element `at` on
            y = torch.cat([torch.zeros(at, dtype=y.dtype, device=DEV), y.reshape(-1)])
            up = torch.cat([torch.ones(at, dtype=up.dtype, device=DEV), up.reshape(-1)])
        return [y.detach()[at:].view(do.shape) if joined else y.detach(), *torch.autograd.grad(y, leaves, up)]

    want = step(lambda x: x.to(DEV), False)
    got = step(lambda x: _sliced(x, at), True)
    assert tsa.tsa_last_device_status() == 0
    for x, y in zip(got, want):
        assert torch.equal(x, y)
