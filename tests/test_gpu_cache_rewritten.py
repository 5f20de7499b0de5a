"""Calls that follow at once on inputs that the device rewrites between them, nothing waited for: queries, positions,
lengths, counts, page tables and schedules as the call before them left them, to the bit of what separate calls give."""
import pytest
import torch

import topology_scheduled_gb300 as tsa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _new(*shape, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


@pytest.mark.parametrize("D,B,HK", [(64, 2, 1), (128, 40, 4)])
def test_tokens_with_everything_rewritten(D, B, HK):
    page, steps, H, cap = 16, 120, 2 * HK, 256
    f = tsa.rotary_frequencies(D)
    pages = B * cap // page
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(1, cap + 1, (steps, B), generator=g, dtype=torch.int32).to(DEV)
    counts = torch.randint(0, 2, (steps, B), generator=g, dtype=torch.int32).to(DEV)
    tables = torch.stack([torch.randperm(pages, generator=g).reshape(B, -1).int() for _ in range(steps)]).to(DEV)
    lists = torch.stack([torch.stack([torch.randperm(4, generator=g)[:2].sort().values for _ in range(B)]).int() for _ in range(steps)]).to(DEV)
    starts = torch.stack([2 * torch.arange(B + 1) if i % 2 else torch.arange(B + 1) for i in range(steps)]).int().to(DEV)
    x = [_new(steps, B, n, 1, D, seed=i) for i, n in enumerate((H, HK, HK))]
    kc0, vc0 = _new(pages, HK, page, D, seed=5), _new(pages, HK, page, D, seed=6)

    def run(wait):
        kc, vc = kc0.clone(), vc0.clone()
        now = [t[0].clone() for t in (*x, lens, counts, tables, lists, starts)]
        got = []
        for i in range(steps):
            for to, t in zip(now, (*x, lens, counts, tables, lists, starts)):
                to.copy_(t[i])
                wait()
            q, k, v, n, c, table, blocks, ptr = now
            one = tsa.tsa_paged_append(q, k, v, kc, vc, table, n, c, f, out=q)
            wait()
            got.append(tsa.tsa_paged_attention_decode(one[:, :, 0], kc, vc, table, n))
            wait()
            got.append(tsa.tsa_paged_attention_decode(one[:, :, 0], kc, vc, table, n, ptr, blocks.flatten()))
            wait()
        torch.cuda.synchronize()
        return [*got, kc, vc]

    want = run(torch.cuda.synchronize)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(run(lambda: None), want))
    assert tsa.tsa_last_device_status() == 0


def test_positions_rewritten_in_place():
    """One token's positions, counted up on the device between rotations of many heads in place."""
    f = [0.3, 0.2, 1.0, 0.7] * 2
    x = _new(3, 64, 5, 16, seed=1)
    pos = _ints([[1000 * b + s for s in range(5)] for b in range(3)])

    def run(wait):
        y, p = x.clone(), pos.clone()
        got = []
        for _ in range(200):
            tsa.tsa_rotary(y, None, f, p, out=y)
            wait()
            got.append(tsa.tsa_rotary(x, None, f, p))
            wait()
            p.add_(1)
            wait()
        return [*got, y]

    want = run(torch.cuda.synchronize)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(run(lambda: None), want))
