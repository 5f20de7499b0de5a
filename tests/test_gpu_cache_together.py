"""Rotary positions, the paged cache and its attention used together, beside the scheduled attention: a layer's
prompt and the tokens after it, a training step, captured graphs, streams, offsets past 32 bits, refusals."""
import pytest
import torch

import topology_scheduled_gb300 as tsa
from topology_scheduled_gb300 import autograd
from _cache import U, attention, close, gathered, page_lists, rotated

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _normal(*shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
def test_a_prompt_and_the_tokens_after_it(interleaved, dtype):
    """Ragged prompts are appended in one call, padded behind; then tokens one by one, each appended and answered,
    for all keys and for a schedule's blocks. Every step meets the 64-bit form over the cache, and the prompt's last
    token meets the scheduled attention of the prompt."""
    B, H, HK, D, page, block = 3, 4, 4, 64, 32, 64
    prompts, steps = [150, 64, 3], 5
    T = max(prompts)
    f = tsa.rotary_frequencies(48, 1000.0, scaling="ramp", factor=2.0, original_length=128)
    mag = tsa.rotary_magnitude(2.0)
    q, k, v = (_normal(B, n, T + steps, D, dtype=dtype, seed=i).to(DEV) for i, n in enumerate((H, HK, HK)))
    table, pages = page_lists([n + steps for n in prompts], page, seed=4)
    kc = torch.full((pages, HK, page, D), float("nan"), dtype=dtype, device=DEV)
    vc, gtable = kc.clone(), table.to(DEV)
    out = tsa.tsa_paged_append(q[:, :, :T], k[:, :, :T], v[:, :, :T], kc, vc, gtable, _ints(prompts), _ints(prompts), f,
                               interleaved=interleaved, magnitude=mag)
    # the same rotation as tsa_rotary's, whose rows the scheduled attention takes
    rq, rk = tsa.tsa_rotary(q[:, :, :T], k[:, :, :T], f, interleaved=interleaved, magnitude=mag)
    for b, n in enumerate(prompts):
        assert torch.equal(out[b, :, :n], rq[b, :, :n]) and bool((out[b, :, n:] == 0).all())
        assert torch.equal(gathered(kc, table[b], n), rk[b, :, :n])
        assert torch.equal(gathered(vc, table[b], n), v[b, :, :n])
    for step in range(-1, steps):
        lens = [n + step + 1 for n in prompts]
        if step < 0:  # the prompt's last token, again
            one = torch.stack([out[b, :, n - 1] for b, n in enumerate(prompts)])
        else:
            at = [torch.stack([x[b, :, n + step] for b, n in enumerate(prompts)])[:, :, None] for x in (q, k, v)]
            one = tsa.tsa_paged_append(*at, kc, vc, gtable, _ints(lens), None, f, interleaved=interleaved, magnitude=mag)[:, :, 0]
            for b, n in enumerate(lens):
                close(one[b][:, None], *rotated(at[0][b], [n - 1], f, interleaved, mag), "Q")
        rows = [[j for j in range(-(-n // block)) if j != 1] for n in lens]
        ptr = [0]
        for r in rows:
            ptr.append(ptr[-1] + len(r))
        for lists in ((None, None), (_ints(ptr), _ints([j for r in rows for j in r]))):
            o = tsa.tsa_paged_attention_decode(one.contiguous(), kc, vc, gtable, _ints(lens), *lists, block=block)
            for b, n in enumerate(lens):
                keep = torch.arange(n)
                keep = keep if lists[0] is None else keep[keep // block != 1]
                K, V = (gathered(x, table[b], n)[:, keep.to(DEV)] for x in (kc, vc))
                want, bound = attention(one[b], K, V, H // HK, D ** -0.5, dtype)
                close(o[b], want, bound, f"step {step}, sequence {b}")
                if step < 0 and lists[0] is None:
                    rp, ci = tsa.tsa_dense_causal_csr(n, block)
                    full = tsa.tsa_scheduled_attention(*(x[b, :, :n].contiguous() for x in (rq, rk, v)), rp, ci)
                    # that kernel rounds its weights
                    top = V.double().abs().amax(1).cpu()
                    close(full[:, -1], want, bound + 2 * U[dtype] * top, "scheduled")
    assert tsa.tsa_last_device_status() == 0
    unused = set(range(pages)) - set(table[table >= 0].tolist())
    for i in unused:
        assert bool(torch.isnan(kc[i]).all()) and bool(torch.isnan(vc[i]).all())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_training_step(dtype):
    """A projection's Q and K rotated and through the scheduled attention; gradients at the projection against the
    64-bit form's, and the rotation's own share bit for bit."""
    B, H, S, D = 2, 3, 130, 64
    f = tsa.rotary_frequencies(D, 500.0)
    x = [_normal(B, S, H, D, dtype=dtype, seed=i).to(DEV).requires_grad_() for i in range(3)]
    g = _normal(B, H, S, D, dtype=dtype, seed=9).to(DEV)
    rp, ci = tsa.tsa_dense_causal_csr(S, 64)
    q, k, v = (t.transpose(1, 2) for t in x)
    rq, rk = autograd.rotary(q, k, f)
    rq.retain_grad()
    rk.retain_grad()
    out = autograd.scheduled_attention(rq, rk, v, rp, ci)
    out.backward(g)
    assert all(t.grad.shape == t.shape for t in x)
    for leaf, r in ((x[0], rq), (x[1], rk)):
        assert torch.equal(leaf.grad, tsa.tsa_rotary(r.grad, None, f, inverse=True).transpose(1, 2))
    # 64 bits, from the rotated rows as they were rounded
    a, b, c = (t.detach().cpu().double().requires_grad_() for t in (rq, rk, v))
    z = a @ b.transpose(2, 3) * D ** -0.5
    P = torch.softmax(z.masked_fill(~torch.ones(S, S, dtype=torch.bool).tril(), -float("inf")), -1)
    (P @ c).backward(g.cpu().double())
    for leaf, want in ((x[0], a.grad), (x[1], b.grad)):
        for i in range(B):
            y, _ = rotated(want[i], range(S), f, inverse=True)
            off = (leaf.grad.transpose(1, 2)[i].cpu().double() - y).norm() / y.norm()
            # P, dS, their products' results and the rotation's are rounded (4 roundings, adding up at worst), and
            # Delta comes from a rounded output: 8 of them leave room for its share
            assert float(off) <= 8 * U[dtype], float(off)


def test_captured_and_replayed():
    """A token's append and attention in a graph, replayed as the sequences grow, beside a second graph."""
    B, H, HK, D, page = 2, 8, 2, 128, 16
    most = 600
    f = tsa.rotary_frequencies(D)
    table, pages = page_lists([most] * B, page, seed=1)
    gtable = table.to(DEV)
    steps = 4
    q, k, v = (_normal(steps, B, n, 1, D, dtype=torch.bfloat16, seed=i).to(DEV) for i, n in enumerate((H, HK, HK)))
    kc0, vc0 = (_normal(pages, HK, page, D, dtype=torch.bfloat16, seed=i).to(DEV) for i in (7, 8))

    def state():
        return [x[0].clone() for x in (q, k, v)] + [kc0.clone(), vc0.clone(), _ints([500, 3])]

    def token(s):
        one = tsa.tsa_paged_append(*s[:5], gtable, s[5], None, f)
        return tsa.tsa_paged_attention_decode(one[:, :, 0], *s[3:5], gtable, s[5])

    def long(s):  # one sequence, split in parts: it has a workspace
        return tsa.tsa_paged_attention_decode(*s)

    n = 40000
    ltable, lpages = page_lists([n], 64, seed=2)
    l = [_normal(1, 1, 64, dtype=torch.float16, seed=1).to(DEV), *(_normal(lpages, 1, 64, 64, dtype=torch.float16, seed=i).to(DEV)
                                                                  for i in (2, 3)), ltable.to(DEV), _ints([n])]
    assert tsa.tsa_paged_attention_decode_workspace_bytes(1, 1, 1, 64, 64, ltable.shape[1]) > 0
    want_long = long(l)
    eager, captured = state(), state()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        token(state())
        long(l)
    torch.cuda.synchronize()
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(one):
        out = token(captured)
    with torch.cuda.graph(two):
        out_long = long(l)
    for i in range(steps):
        for s in (eager, captured):
            for to, x in zip(s[:3], (q, k, v)):
                to.copy_(x[i])
            s[5] += 1
        want = token(eager)
        two.replay()
        one.replay()
        two.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(out_long, want_long)
        for a, b in zip(eager[3:5], captured[3:5]):
            assert torch.equal(a, b)
    assert tsa.tsa_last_device_status() == 0


def test_a_captured_training_step():
    f = tsa.rotary_frequencies(64)
    q = _normal(1, 2, 40, 64, dtype=torch.float16, seed=1).to(DEV).requires_grad_()
    k = _normal(1, 2, 40, 64, dtype=torch.float16, seed=2).to(DEV).requires_grad_()
    g = _normal(1, 2, 40, 64, dtype=torch.float16, seed=3).to(DEV)

    def step():
        a, b = autograd.rotary(q, k, f)
        return torch.autograd.grad([a, b], [q, k], [g, g])

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    g.mul_(-2)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, -2 * b)


def test_on_another_stream():
    """Inputs made on the stream that the calls are asked to run on, while the current one is busy elsewhere."""
    B, H, D, page = 2, 4, 64, 16
    f = tsa.rotary_frequencies(D)
    table, pages = page_lists([200, 90], page, seed=5)
    gtable = table.to(DEV)
    base = [_normal(B, H, 1, D, dtype=torch.float16, seed=i).to(DEV) for i in range(3)]
    kc, vc = (_normal(pages, H, page, D, dtype=torch.float16, seed=i).to(DEV) for i in (5, 6))
    lens = _ints([200, 90])
    kc1, vc1 = kc.clone(), vc.clone()
    rot = tsa.tsa_rotary(base[0], base[1], f)
    one = tsa.tsa_paged_append(*base, kc1, vc1, gtable, lens, None, f)
    want = tsa.tsa_paged_attention_decode(one[:, :, 0], kc1, vc1, gtable, lens)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = torch.randn((4096, 4096), device=DEV)
    for _ in range(10):
        busy = busy @ busy * 1e-2
    got_rot = tsa.tsa_rotary(base[0], base[1], f, stream=s)
    got_one = tsa.tsa_paged_append(*base, kc, vc, gtable, lens, None, f, stream=s)
    got = tsa.tsa_paged_attention_decode(got_one[:, :, 0], kc, vc, gtable, lens, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(got_one, one) and torch.equal(kc, kc1)
    assert all(torch.equal(a, b) for a, b in zip(got_rot, rot))


def test_the_order_of_thread_blocks_changes_nothing():
    table, pages = page_lists([70000, 65000], 64, seed=5)
    args = [_normal(2, 4, 128, dtype=torch.bfloat16, seed=1).to(DEV),
            *(torch.randn((pages, 2, 64, 128), device=DEV, dtype=torch.bfloat16) for _ in range(2)), table.to(DEV),
            _ints([70000, 65000])]
    first = tsa.tsa_paged_attention_decode(*args)
    for _ in range(5):
        assert torch.equal(tsa.tsa_paged_attention_decode(*args), first)


def test_pages_past_2_to_the_31_elements():
    HK, page, D = 8, 256, 128
    one = HK * page * D
    pages = (1 << 31) // one + 40
    kc = torch.zeros((pages, HK, page, D), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    lengths = [700, 300]
    table = torch.tensor([[pages - 1, pages - 33, 5], [pages - 7, pages - 2, -1]], dtype=torch.int32)
    gtable = table.to(DEV)
    f = tsa.rotary_frequencies(D)
    q, k, v = (_normal(2, n, 700, D, dtype=torch.bfloat16, seed=i).to(DEV) for i, n in enumerate((16, HK, HK)))
    out = tsa.tsa_paged_append(q, k, v, kc, vc, gtable, _ints(lengths), _ints(lengths), f)
    for b, n in enumerate(lengths):
        some = [0, 1, 255, 256, n - 1]
        close(gathered(kc, table[b], n)[:, some], *rotated(k[b][:, some], some, f), "K")
        assert torch.equal(gathered(vc, table[b], n), v[b, :, :n])
    last = torch.stack([out[b, :, n - 1] for b, n in enumerate(lengths)])
    o = tsa.tsa_paged_attention_decode(last, kc, vc, gtable, _ints(lengths))
    for b, n in enumerate(lengths):
        close(o[b], *attention(last[b], gathered(kc, table[b], n), gathered(vc, table[b], n), 2, D ** -0.5, torch.bfloat16))
    used = sorted(int(x) for x in table.flatten() if x >= 0)
    assert float(kc[[i for i in (0, 1, 4, 6, pages - 3, pages - 34) if i not in used]].abs().max()) == 0
    assert tsa.tsa_last_device_status() == 0


def test_rows_past_2_to_the_31_elements():
    H, S, D = 64, 270000, 128
    x = torch.zeros((1, S, H, D), dtype=torch.float16, device=DEV)
    f = tsa.rotary_frequencies(D)
    some = [0, 1, 262143, 262144, S - 1]
    rows = _normal(1, H, len(some), D, dtype=torch.float16, seed=1)
    x[:, some] = rows.transpose(1, 2).to(DEV)
    out = tsa.tsa_rotary(x.transpose(1, 2), None, f)
    assert out.numel() > 1 << 31
    close(out[:, :, some], *rotated(rows, some, f))
    assert float(out[0, 63, 200000:200050].abs().max()) == 0


def test_refusals():
    f = tsa.rotary_frequencies(64)
    x = torch.zeros((2, 4, 8, 64), dtype=torch.float16, device=DEV)
    kc = torch.zeros((5, 4, 16, 64), dtype=torch.float16, device=DEV)
    table, lens = _ints([[0, 1], [2, 3]]), _ints([8, 8])
    q = x[:, :, 0].contiguous()
    wide = torch.zeros((2, 4, 8, 128), dtype=torch.float16, device=DEV)
    value = [
        lambda: tsa.tsa_rotary(x[0], x, f), lambda: tsa.tsa_rotary(x, x.bfloat16(), f), lambda: tsa.tsa_rotary(x, x[:, :, :4], f),
        lambda: tsa.tsa_rotary(x, x[:1], f), lambda: tsa.tsa_rotary(wide[..., ::2], None, f),
        lambda: tsa.tsa_rotary(x, None, f, _ints([0] * 7)), lambda: tsa.tsa_rotary(x, None, f, _ints([0] * 8).long()),
        lambda: tsa.tsa_rotary(x, None, f, _ints([0] * 8).cpu()), lambda: tsa.tsa_rotary(x, None, f, out=x[:, :2]),
        lambda: tsa.tsa_rotary(x, None, f, out_k=x), lambda: tsa.tsa_rotary(x, None, torch.ones(32, device=DEV)),
        lambda: tsa.tsa_paged_append(x, x, x, kc, kc, table, lens), lambda: tsa.tsa_paged_append(None, x, x, kc, kc, table, lens, out=x),
        lambda: tsa.tsa_paged_append(None, x, x[:, :2], kc, kc, table, lens),
        lambda: tsa.tsa_paged_append(None, x, x, kc[..., :32], kc, table, lens),
        lambda: tsa.tsa_paged_append(None, x, x, kc, kc.transpose(1, 2), table, lens),
        lambda: tsa.tsa_paged_append(None, x, x, kc, kc, table[:1], lens), lambda: tsa.tsa_paged_append(None, x, x, kc, kc, table, lens[:1]),
        lambda: tsa.tsa_paged_append(None, x, x, kc, kc, table, lens, lens[:1]),
        lambda: tsa.tsa_paged_attention_decode(x, kc, kc, table, lens), lambda: tsa.tsa_paged_attention_decode(q.bfloat16(), kc, kc, table, lens),
        lambda: tsa.tsa_paged_attention_decode(q, kc, kc[:, :2], table, lens), lambda: tsa.tsa_paged_attention_decode(q, kc, kc, table.t(), lens),
        lambda: tsa.tsa_paged_attention_decode(q, kc, kc, table, lens, _ints([0, 1, 2])),
        lambda: tsa.tsa_paged_attention_decode(q, kc, kc, table, lens, _ints([0, 1]), _ints([0]))]
    for i, call in enumerate(value):
        with pytest.raises(ValueError):
            call()
            print("taken:", i)
    off = torch.zeros(2 * 4 * 8 * 64 + 8, dtype=torch.float16, device=DEV)[1:-7].reshape(2, 4, 8, 64)  # off a 16-byte boundary
    odd = torch.zeros((2, 4, 8, 68), dtype=torch.float16, device=DEV)[..., :64]                        # rows 136 bytes apart
    status = [
        (1, lambda: tsa.tsa_rotary(off, None, f)), (1, lambda: tsa.tsa_rotary(odd, None, f)), (1, lambda: tsa.tsa_rotary(x, x, f, out=x)),
        (1, lambda: tsa.tsa_rotary(x, None, f, out=x[:, :, :1].expand(2, 4, 8, 64))), (2, lambda: tsa.tsa_rotary(x, None, [1.0] * 4)),
        (2, lambda: tsa.tsa_rotary(x, None, [1.0] * 40)), (1, lambda: tsa.tsa_rotary(x, None, [float("nan")] * 8)),
        (1, lambda: tsa.tsa_paged_append(None, x, x, kc, kc, table, lens)),
        (2, lambda: tsa.tsa_paged_append(None, x, x, kc[:, :, :8].contiguous(), kc[:, :, :8].contiguous(), table, lens)),
        (1, lambda: tsa.tsa_paged_attention_decode(q[:, :3].contiguous(), kc, kc, table, lens)),
        (2, lambda: tsa.tsa_paged_attention_decode(q, kc, kc, table, lens, _ints([0, 1, 2]), _ints([0, 0]), block=16)),
        (1, lambda: tsa.tsa_paged_attention_decode(q, kc, kc, table, lens, scale=0.0)),
        (1, lambda: tsa.tsa_paged_attention_decode(q, kc, kc, table, lens, out=q))]
    for want, call in status:
        with pytest.raises(tsa.TsaError) as e:
            call()
        assert e.value.status == want
    with pytest.raises(TypeError):
        tsa.tsa_rotary(x.float(), None, f)
    assert tsa.tsa_last_device_status() == 0


def test_several_host_threads():
    """Threads with streams of their own, whose calls differ in size (some with a workspace): each gets what it gets alone."""
    import threading

    f = tsa.rotary_frequencies(64)

    def inputs(i):
        H, HK, n, page = ((4, 4, 300, 16), (8, 1, 30000, 64), (16, 2, 90, 32))[i % 3]
        lengths = [n + i, 5]
        table, pages = page_lists(lengths, page, seed=i)
        x = [_normal(2, h, 1, 64, dtype=torch.float16, seed=10 * i + j).to(DEV) for j, h in enumerate((H, HK, HK))]
        return x, [_normal(pages, HK, page, 64, dtype=torch.float16, seed=50 + 10 * i + j).to(DEV) for j in range(2)], table.to(DEV), \
            _ints(lengths)

    def run(x, caches, table, lens):
        kc, vc = (c.clone() for c in caches)
        q = tsa.tsa_paged_append(*x, kc, vc, table, lens, None, f)
        return tsa.tsa_paged_attention_decode(q[:, :, 0], kc, vc, table, lens), kc, vc

    data = [inputs(i) for i in range(6)]
    alone = [run(*d) for d in data]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        try:
            torch.cuda.set_device(0)
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got = run(*data[i])
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, alone[i])):
                        wrong.append(i)
                        return
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
    assert tsa.tsa_last_device_status() == 0


def test_captured_on_forked_streams():
    """A capture that forks: keys are appended on one stream while queries are rotated on another, and the attention
    waits for both; a copy and a fill stand before and behind. Replayed on new inputs, it gives what the eager calls give."""
    B, H, HK, D, page = 4, 8, 4, 64, 32
    lengths = [333, 70, 1, 128]
    f = tsa.rotary_frequencies(D)
    table, pages = page_lists(lengths, page, seed=6)
    gtable, lens = table.to(DEV), _ints(lengths)
    pos = (lens - 1)[:, None].contiguous()
    kc0, vc0 = (_normal(pages, HK, page, D, dtype=torch.float16, seed=i).to(DEV) for i in (1, 2))

    def inputs(seed):
        return [_normal(B, n, 1, D, dtype=torch.float16, seed=seed + i).to(DEV) for i, n in enumerate((H, HK, HK))]

    def eager(x):
        kc, vc = kc0.clone(), vc0.clone()
        tsa.tsa_paged_append(None, x[1], x[2], kc, vc, gtable, lens, None, f)
        q = tsa.tsa_rotary(x[0], None, f, pos)
        return tsa.tsa_paged_attention_decode(q[:, :, 0], kc, vc, gtable, lens)

    held, kc, vc = inputs(100), kc0.clone(), vc0.clone()
    kept = torch.empty((B, H, D), dtype=torch.float16, device=DEV)
    eager(held)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        kc.copy_(kc0)
        vc.copy_(vc0)
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            tsa.tsa_paged_append(None, held[1], held[2], kc, vc, gtable, lens, None, f)
        q = tsa.tsa_rotary(held[0], None, f, pos)
        main.wait_stream(side)
        out = tsa.tsa_paged_attention_decode(q[:, :, 0], kc, vc, gtable, lens)
        kept.copy_(out)
        out.zero_()
    for seed in (200, 300, 400):
        x = inputs(seed)
        want = eager(x)
        for a, b in zip(held, x):
            a.copy_(b)
        for _ in range(3):
            kept.fill_(7)
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept, want)
    assert tsa.tsa_last_device_status() == 0


def test_back_to_back_on_one_buffer():
    """Calls that follow at once, each reading what the one before wrote (a kernel is set up before its predecessor
    has ended): a row rotated a hundred times in place, and a cache's one slot rewritten between its readers."""
    f = [0.25] * 8
    x = _normal(1, 64, 200, 64, dtype=torch.float16, seed=1).to(DEV)
    want = x.clone()
    for _ in range(100):
        want = tsa.tsa_rotary(want, None, f)
        torch.cuda.synchronize()
    for _ in range(100):
        tsa.tsa_rotary(x, None, f, out=x)
    assert torch.equal(x, want)
    kc = torch.zeros((1, 1, 16, 64), dtype=torch.float16, device=DEV)
    vc = torch.zeros_like(kc)
    table, lens = _ints([[0]]), _ints([1])
    q = torch.ones((1, 1, 64), dtype=torch.float16, device=DEV)
    values = torch.arange(1, 501, device=DEV).half()[:, None, None, None, None].expand(500, 1, 1, 1, 64).contiguous()
    got = []
    for i in range(500):
        tsa.tsa_paged_append(None, values[i], values[i], kc, vc, table, lens)
        got.append(tsa.tsa_paged_attention_decode(q, kc, vc, table, lens))
    assert torch.equal(torch.cat(got)[:, 0], values[:, 0, 0, 0])
