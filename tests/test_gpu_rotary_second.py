"""A rotation's backward pass that is differentiated itself takes any upstream gradient that the plain one takes."""
import pytest
import torch

import topology_scheduled_gb300 as tsa
from topology_scheduled_gb300 import autograd
from _cache import close, rotated

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _normal(*shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def _gradients(B, H, S, D, dtype):
    """An expanded gradient, one of transposed rows, one that starts off a 16-byte boundary."""
    wide = _normal(B, H, S, D + 1, dtype=dtype, seed=4).to(DEV)
    return {"expanded": torch.ones((), dtype=dtype, device=DEV).expand(B, H, S, D),
            "transposed": _normal(B, H, D, S, dtype=dtype, seed=3).to(DEV).transpose(2, 3), "offset": wide[..., 1:]}


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("kind", ["expanded", "transposed", "offset"])
def test_gradients_of_any_layout(kind, dtype):
    B, H, S, D = 2, 3, 6, 64
    f = tsa.rotary_frequencies(48)
    q, k = (_normal(B, h, S, D, dtype=dtype, seed=h).to(DEV).requires_grad_() for h in (H, 1))
    g = _gradients(B, H, S, D, dtype)[kind].detach().requires_grad_()
    v = _normal(B, H, S, D, dtype=dtype, seed=9).to(DEV)
    out, out_k = autograd.rotary(q, k, f, None, True, 1.5)
    dq, = torch.autograd.grad(out, [q], g, create_graph=True)
    close(dq, *rotated(g, range(S), f, True, 1.5, inverse=True))
    dg, = torch.autograd.grad(dq, [g], v)
    close(dg, *rotated(v, range(S), f, True, 1.5))
    out, out_k = autograd.rotary(q, k, f, None, True, 1.5)
    dq, dk = torch.autograd.grad([out, out_k], [q, k], [g, g[:, :1]], create_graph=True)
    close(dq, *rotated(g, range(S), f, True, 1.5, inverse=True))
    close(dk, *rotated(g[:, :1], range(S), f, True, 1.5, inverse=True))


def test_a_penalty_on_a_gradient():
    """The gradient of |d sum(rotary(q) rotary(q)) / dq|^2, whose upstream gradients are sums' expanded ones."""
    S, D = 5, 64
    f = tsa.rotary_frequencies(D)
    q = _normal(1, 2, S, D, dtype=torch.bfloat16, seed=1).to(DEV).requires_grad_()
    out = autograd.rotary(q, None, f)
    dq, = torch.autograd.grad(out.sum(), [q], create_graph=True)
    ones, bound = rotated(torch.ones(1, 2, S, D), range(S), f, inverse=True)
    close(dq, ones, bound)
    out = autograd.rotary(q, None, f)
    dq, = torch.autograd.grad((out * out).sum(), [q], create_graph=True)
    # 2 R^T R 1 = 2.  R 1 is at most 1.42 and rounded by 1.42 2^-8, which twice R^T makes at most 1.42 times 2.84 2^-8 = 4.1 2^-8;
    # the result's rounding adds 2 x 2^-8
    dq.sum().backward()
    assert bool(((q.grad.double() - 2).abs() <= 7 * 2.0 ** -8).all())
