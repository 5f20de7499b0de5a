"""Rotary positions on the GPU against the 64-bit form: layouts, parts of the head, positions near and far,
views, in place, gradients."""
import math

import pytest
import torch

import topology_scheduled_gb300 as tsa
from topology_scheduled_gb300 import autograd
from _cache import close, rotated

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _normal(*shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,HK,S,D,R", [(1, 1, 1, 1, 64, 64), (2, 3, 1, 5, 64, 32), (1, 32, 8, 33, 128, 128),
                                          (3, 5, 5, 7, 128, 16), (1, 2, 1, 40, 64, 48), (2, 17, 3, 3, 256, 256),
                                          (1, 1, 2, 19, 16, 16), (2, 2, 2, 65, 96, 96), (1, 4, 1, 700, 128, 64)])
def test_against_the_definition(B, H, HK, S, D, R, interleaved, dtype):
    q, k = _normal(B, H, S, D, dtype=dtype, seed=1), _normal(B, HK, S, D, dtype=dtype, seed=2)
    f = tsa.rotary_frequencies(R, 10000.0)
    out, out_k = tsa.tsa_rotary(q.to(DEV), k.to(DEV), f, interleaved=interleaved, magnitude=1.25)
    assert out.is_contiguous() and out_k.is_contiguous()
    for name, got, x in (("Q", out, q), ("K", out_k, k)):
        close(got, *rotated(x, range(S), f, interleaved, 1.25), name)
        assert torch.equal(got[..., R:].cpu(), x[..., R:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_positions(interleaved):
    """Far, negative and repeated positions, per batch and shared; frequencies from whole turns to none."""
    S, D = 12, 64
    x = _normal(2, 3, S, D, dtype=torch.float16, seed=3)
    f = [65536.0, -3.5, 2 * math.pi, 1.0, 0.3, 1e-3, 1e-9, 0.0, -1e-9, -0.0, -65536.0, 1e-300, -0.3, 4096.25, -1e-5, 1e-16]
    f += list(tsa.rotary_frequencies(32, 1e6))
    rows = [[0, 1, -1, 2, 1 << 20, 1 << 30, (1 << 31) - 1, -(1 << 31), 131071, 5, 5, -77777],
            [1000003 * i for i in range(S)]]
    pos = torch.tensor(rows, dtype=torch.int32, device=DEV)
    out = tsa.tsa_rotary(x.to(DEV), None, f, pos, interleaved=interleaved)
    for b in range(2):
        close(out[b], *rotated(x[b], rows[b], f, interleaved), f"batch {b}")
    out = tsa.tsa_rotary(x.to(DEV), None, f, pos[0].contiguous(), interleaved=interleaved)
    for b in range(2):
        close(out[b], *rotated(x[b], rows[0], f, interleaved), f"shared, batch {b}")


def test_many_heads():
    x = _normal(1, 30000, 1, 16, dtype=torch.bfloat16, seed=5)
    f = tsa.rotary_frequencies(16, 100.0)
    out = tsa.tsa_rotary(x.to(DEV), x[:, :7].to(DEV), f, torch.tensor([77], dtype=torch.int32, device=DEV))
    close(out[0], *rotated(x, [77], f))
    close(out[1], *rotated(x[:, :7], [77], f))


def test_inverse_undoes():
    x = _normal(1, 4, 50, 128, dtype=torch.float16, seed=4).to(DEV)
    f = tsa.rotary_frequencies(128)
    there = tsa.tsa_rotary(x, None, f, magnitude=2.0)
    want, bound = rotated(there.cpu(), range(50), f, False, 0.5, inverse=True)
    back = tsa.tsa_rotary(there, None, f, magnitude=0.5, inverse=True)
    close(back, want, bound)
    # rounding there (2^-11 of each side of a pair) and back
    pair = x.double().abs() + x.double().abs().roll(64, -1)
    assert bool(((back - x).abs().double() <= 2.0 ** -10 * pair + 2.0 ** -22).all())


def _joint(dtype, seed=5, B=2, S=37, H=4, HK=2, D=64):
    """Q, K, V heads side by side in one projection [B, S, (H + 2 HK) D], as views."""
    x = _normal(B, S, H + 2 * HK, D, dtype=dtype, seed=seed)
    return x, lambda y: (y[:, :, :H].transpose(1, 2), y[:, :, H:H + HK].transpose(1, 2), y[:, :, H + HK:].transpose(1, 2))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_views_and_in_place(dtype):
    x, parts = _joint(dtype)
    f = tsa.rotary_frequencies(64)
    q, k, v = parts(x)
    whole = x.to(DEV)
    gq, gk, gv = parts(whole)
    out, out_k = tsa.tsa_rotary(gq, gk, f)
    close(out, *rotated(q, range(37), f))
    close(out_k, *rotated(k, range(37), f))
    assert torch.equal(whole.cpu(), x)
    # into a view of another layout, whose other elements stay
    wide = torch.full((2, 37, 4, 80), 7.0, dtype=dtype, device=DEV)
    tsa.tsa_rotary(gq, None, f, out=wide[..., 8:72].transpose(1, 2))
    assert torch.equal(wide[..., 8:72].transpose(1, 2), out)
    assert bool((wide[..., :8] == 7).all()) and bool((wide[..., 72:] == 7).all())
    # the joint projection's Q and K heads in place, V's left alone
    a, b = tsa.tsa_rotary(gq, gk, f, out=gq, out_k=gk)
    assert a.data_ptr() == gq.data_ptr() and torch.equal(gq, out) and torch.equal(gk, out_k)
    assert torch.equal(gv.cpu(), v)
    # an input whose heads are one
    one = _normal(2, 1, 37, 64, dtype=dtype, seed=9)
    many = tsa.tsa_rotary(one.to(DEV).expand(2, 5, 37, 64), None, f)
    close(many, *rotated(one.expand(2, 5, 37, 64), range(37), f))


def test_what_is_not_finite_stays_in_its_pair():
    x = _normal(1, 2, 3, 64, dtype=torch.bfloat16, seed=6)
    x[0, 0, 1, 5], x[0, 1, 2, 40] = float("nan"), float("inf")
    out = tsa.tsa_rotary(x.to(DEV), None, tsa.rotary_frequencies(64)).cpu()
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[0, 0, 1, [5, 37]] = True
    want[0, 1, 2, [8, 40]] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens_first", [False, True])
def test_gradients(tokens_first, interleaved, dtype):
    B, S, H, HK, D, R = 2, 29, 4, 2, 64, 32
    f = tsa.rotary_frequencies(R, scaling="linear", factor=4.0)
    pos = torch.tensor([[3 * i + 100 * b for i in range(S)] for b in range(B)], dtype=torch.int32, device=DEV)

    def leaf(h, seed):
        shape = (B, S, h, D) if tokens_first else (B, h, S, D)
        return _normal(*shape, dtype=dtype, seed=seed).to(DEV).requires_grad_()

    lq, lk = leaf(H, 1), leaf(HK, 2)
    q, k = (x.transpose(1, 2) if tokens_first else x for x in (lq, lk))
    out, out_k = autograd.rotary(q, k, f, pos, interleaved, 1.5)
    gq, gk = _normal(B, H, S, D, dtype=dtype, seed=3).to(DEV), _normal(B, HK, S, D, dtype=dtype, seed=4).to(DEV)
    dq, dk = torch.autograd.grad([out, out_k], [lq, lk], [gq, gk])
    assert dq.is_contiguous() and dk.is_contiguous()  # in their leaves' layout
    for x, got, g in ((q, dq, gq), (k, dk, gk)):
        got = got.transpose(1, 2) if tokens_first else got
        for b in range(B):
            want, bound = rotated(g[b], pos[b].tolist(), f, interleaved, 1.5, inverse=True)
            close(got[b], want, bound, "gradient")
    # against differences of the 64-bit form: <g, d out / d x> along a direction
    e = _normal(S, D, dtype=torch.float64, seed=8)
    y0, _ = rotated(q[0, 0], pos[0].tolist(), f, interleaved, 1.5)
    y1, _ = rotated(q[0, 0].detach().cpu().double() + e, pos[0].tolist(), f, interleaved, 1.5)
    by_difference = float((gq[0, 0].cpu().double() * (y1 - y0)).sum())
    want, bound = rotated(gq[0, 0], pos[0].tolist(), f, interleaved, 1.5, inverse=True)
    assert abs(float((want * e).sum()) - by_difference) <= 1e-10 * float((want.abs() * e.abs()).sum())


def test_gradients_of_one_and_of_views():
    """Only one of Q and K wants a gradient; the upstream gradient is expanded, or starts off a 16-byte boundary."""
    B, S, H, D = 1, 10, 2, 64
    f = tsa.rotary_frequencies(D)
    q = _normal(B, H, S, D, dtype=torch.float16, seed=1).to(DEV).requires_grad_()
    k = _normal(B, H, S, D, dtype=torch.float16, seed=2).to(DEV).requires_grad_()
    ones, _ = rotated(torch.ones(B, H, S, D), range(S), f, inverse=True)
    bound = 2.0 ** -20 * torch.ones_like(ones)
    out, out_k = autograd.rotary(q, k.detach(), f)
    out.sum().backward()
    close(q.grad, ones, bound)
    out, out_k = autograd.rotary(q.detach(), k, f)
    out_k.sum().backward()
    close(k.grad, ones, bound)
    out, out_k = autograd.rotary(q, k, f)
    dk, = torch.autograd.grad(out_k.sum(), [k])
    close(dk, ones, bound)
    alone = autograd.rotary(q, None, f)
    wide = _normal(B, H, S, D + 1, dtype=torch.float16, seed=3).to(DEV)
    dq, = torch.autograd.grad(alone, [q], wide[..., 1:])
    close(dq, *rotated(wide[..., 1:], range(S), f, inverse=True))


def test_positions_changed_before_the_backward_are_noticed():
    q = _normal(1, 1, 4, 64, dtype=torch.float16, seed=1).to(DEV).requires_grad_()
    pos = torch.arange(4, dtype=torch.int32, device=DEV)
    out = autograd.rotary(q, None, tsa.rotary_frequencies(64), pos)
    pos += 1
    with pytest.raises(RuntimeError):
        out.sum().backward()


@pytest.mark.parametrize("interleaved", [False, True])
def test_second_gradients(interleaved):
    """The backward pass is a rotation, and has a gradient of its own: <v, dQ(g)> has the gradient R v by g."""
    f = tsa.rotary_frequencies(64)
    q = _normal(1, 2, 6, 64, dtype=torch.float16, seed=1).to(DEV).requires_grad_()
    g = _normal(1, 2, 6, 64, dtype=torch.float16, seed=2).to(DEV).requires_grad_()
    v = _normal(1, 2, 6, 64, dtype=torch.float16, seed=3).to(DEV)
    out = autograd.rotary(q, None, f, None, interleaved, 1.5)
    dq, = torch.autograd.grad(out, [q], g, create_graph=True)
    dg, = torch.autograd.grad(dq, [g], v)
    close(dq, *rotated(g, range(6), f, interleaved, 1.5, inverse=True))
    close(dg, *rotated(v, range(6), f, interleaved, 1.5))
