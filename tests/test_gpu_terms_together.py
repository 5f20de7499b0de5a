"""The attentions with learned score terms as a model uses them: one after the other over a built
schedule, trained and decoded, in CUDA graphs, on other streams, and at sizes past 32-bit offsets."""
import numpy as np
import pytest
import torch

import topology_scheduled_gb300 as tsa
from _terms import U, _close, biased, differential
from test_gpu_biased import DEV, STARTS, _csr, _dev
from test_gpu_decode import _lists, _reference
from topology_scheduled_gb300.autograd import biased_attention, differential_attention

pytestmark = pytest.mark.gpu
GEO = STARTS["geometric"]
INIT = 0.5
BIASED, DIFF = ("dQ", "dK", "dV", "dbias"), ("dQ", "dK", "dV", "dlq1", "dlk1", "dlq2", "dlk2")


def _learned(H, D, dtype, seed, heads=1):
    g = torch.Generator().manual_seed(seed)
    bias = torch.randn((H, len(GEO)), generator=g).to(dtype)
    return bias, [(0.2 * torch.randn((heads, D // 2), generator=g)).to(dtype) for _ in range(4)]


def _rand(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


@pytest.mark.parametrize("B,H,S,D,dtype", [(2, 2, 500, 64, torch.float16), (1, 3, 640, 128, torch.bfloat16)])
def test_two_layers_trained_and_decoded(B, H, S, D, dtype):
    """A biased and a differential layer with a residual between them, over the schedule built from the
    first one's keys.  Each layer is held to its own bounds at the inputs it got; the whole's gradients
    are those of the layers' calls, bit for bit."""
    q, k, v, k2, v2, do = (_rand((B, H, S, D), dtype, 40 + i) for i in range(6))
    bias, lam = _learned(H, D, dtype, 7, H)
    leaves = [x.to(DEV).requires_grad_(True) for x in (q, k, v, bias, k2, v2, *lam)]
    qd, kd, vd, bd, k2d, v2d, *ld = leaves
    rp, ci = tsa.tsa_build_schedule(kd.detach())
    o1 = biased_attention(qd, kd, vd, rp, ci, bd, GEO)
    mid = qd + o1
    out = differential_attention(mid, k2d, v2d, rp, ci, *ld, INIT)
    grads = torch.autograd.grad(out, leaves, do.to(DEV))
    assert tsa.tsa_last_device_status() == 0
    rp_h, ci_h = rp.cpu().numpy(), ci.cpu().numpy()
    # the second layer
    two = differential(mid, k2, v2, rp_h, ci_h, 64, (D / 2) ** -0.5, lam, INIT, do)
    _close(out, *two["O"], "O of the differential layer")
    with torch.no_grad():
        _, o2, lse2 = tsa.tsa_differential_attention_fwd(mid, k2d, v2d, rp, ci, *ld, INIT)
        g2 = tsa.tsa_differential_attention_backward(mid, k2d, v2d, out, o2, do.to(DEV), lse2, rp, ci, *ld, INIT)
        for name, x in zip(DIFF, g2):
            _close(x, *two[name], "differential " + name)
        # the first
        one = biased(q, k, v, rp_h, ci_h, 64, D ** -0.5, bias, GEO, g2[0])
        _close(o1, *one["O"], "O of the biased layer")
        lse1 = tsa.tsa_biased_attention_fwd(qd, kd, vd, rp, ci, bd, GEO)[1]
        g1 = tsa.tsa_biased_attention_backward(qd, kd, vd, o1, g2[0], lse1, rp, ci, bd, GEO)
        for name, x in zip(BIASED, g1):
            _close(x, *one[name], "biased " + name)
        want = [g1[0] + g2[0], g1[1], g1[2], g1[3], *g2[1:]]
    for x, y in zip(grads, want):
        assert torch.equal(x, y)
    # the last token again, against caches longer than the sequence, over the schedule's last row
    cap, nb = S + 77, -(-S // 64)
    caches = [torch.full((B, H, cap, D), float("nan"), dtype=dtype, device=DEV) for _ in range(4)]
    for c, x in zip(caches, (kd, vd, k2d, v2d)):
        c[:, :, :S] = x.detach()
    row = ci_h[rp_h[nb - 1]:rp_h[nb]].tolist()
    lens, lists = torch.full((B,), S, dtype=torch.int32, device=DEV), _lists([row] * B)
    with torch.no_grad():
        last = qd[:, :, -1].contiguous()
        d1 = tsa.tsa_biased_attention_decode(last, *caches[:2], lens, *lists, bd, GEO)
        want, bound = _reference(last.cpu(), k, v, [S] * B, [row] * B, 64, D ** -0.5, bias, GEO)
        _close(d1, want, bound, "biased decode")
        _close(o1[:, :, -1], want, bound + 2 * U[dtype] * v.double().abs().amax(2), "biased forward")
        x = last + d1
        e1, e2 = (torch.exp((a.double() * b.double()).sum(-1)) for a, b in (lam[:2], lam[2:]))
        d2 = tsa.tsa_differential_attention_decode(x, *caches[2:], lens, *lists, *ld, INIT)
        want, bound = _reference(x.cpu(), k2, v2, [S] * B, [row] * B, 64, (D / 2) ** -0.5, lam=e1 - e2 + INIT)
        _close(d2, want, bound, "differential decode")
    assert tsa.tsa_last_device_status() == 0


class Step:
    """Forward, backward and decode of both attentions with every tensor its own, allocated beforehand."""

    def __init__(self, S, D, dtype, seed, block=64):
        self.block = block
        B, H, nb = 1, 2, -(-S // block)
        self.q, self.k, self.v, self.do = (_rand((B, H, S, D), dtype, seed + i).to(DEV) for i in range(4))
        bias, lam = _learned(H, D, dtype, seed)
        self.bias, self.lam = bias.to(DEV), [x.to(DEV) for x in lam]
        self.rp, self.ci = _dev(*_csr("random", S, block, seed))
        new = torch.empty_like
        self.o, self.od, self.o2 = new(self.q), new(self.q), new(self.q)
        self.lse = torch.empty((B * H, S), dtype=torch.float32, device=DEV)
        self.lse2 = torch.empty((2, B * H, S), dtype=torch.float32, device=DEV)
        self.gb = [new(x) for x in (self.q, self.k, self.v, self.bias)]
        self.gd = [new(x) for x in (self.q, self.k, self.v, *self.lam)]
        L = tsa.lib()
        ws = max(L.tsa_biased_attention_backward_workspace_bytes(B * H, S, block, self.ci.numel(), len(GEO)),
                 L.tsa_differential_attention_backward_workspace_bytes(B * H, S, block, self.ci.numel()))
        self.ws = torch.empty(ws, dtype=torch.uint8, device=DEV)
        self.lens = torch.tensor([S], dtype=torch.int32, device=DEV)
        self.lists = _lists([list(range(nb))])
        self.last = self.q[:, :, -1].contiguous()
        self.d1, self.d2 = new(self.last), new(self.last)

    def run(self, stream=None):
        kw = dict(block=self.block, stream=stream)
        args = self.q, self.k, self.v
        tsa.tsa_biased_attention_fwd(*args, self.rp, self.ci, self.bias, GEO, out=self.o, lse=self.lse, **kw)
        tsa.tsa_biased_attention_backward(*args, self.o, self.do, self.lse, self.rp, self.ci, self.bias, GEO,
                                          dq=self.gb[0], dk=self.gb[1], dv=self.gb[2], dbias=self.gb[3],
                                          workspace=self.ws, **kw)
        tsa.tsa_differential_attention_fwd(*args, self.rp, self.ci, *self.lam, INIT, out=self.od, out2=self.o2,
                                           lse=self.lse2, **kw)
        tsa.tsa_differential_attention_backward(*args, self.od, self.o2, self.do, self.lse2, self.rp, self.ci, *self.lam,
                                                INIT, dq=self.gd[0], dk=self.gd[1], dv=self.gd[2],
                                                dlambdas=self.gd[3:], workspace=self.ws, **kw)
        tsa.tsa_biased_attention_decode(self.last, self.k, self.v, self.lens, *self.lists, self.bias, GEO, out=self.d1, **kw)
        tsa.tsa_differential_attention_decode(self.last, self.k, self.v, self.lens, *self.lists, *self.lam, INIT,
                                              out=self.d2, **kw)

    def results(self):
        return [self.o, self.od, self.o2, self.lse, self.lse2, *self.gb, *self.gd, self.d1, self.d2]

    def expect(self):
        self.run()
        torch.cuda.synchronize()
        assert tsa.tsa_last_device_status() == 0
        want = [x.clone() for x in self.results()]
        self.forget()
        return want

    def forget(self):
        for x in self.results():
            x.fill_(7.0)
        torch.cuda.synchronize()

    def check(self, want):
        assert tsa.tsa_last_device_status() == 0
        for i, (x, y) in enumerate(zip(self.results(), want)):
            assert torch.equal(x, y), i


def test_graphs_with_their_own_workspaces_run_at_once():
    """Two captured steps, replayed at the same time on two streams, with inputs changed after capture."""
    steps = [Step(1000, 64, torch.float16, 3), Step(700, 128, torch.bfloat16, 4, block=128)]
    graphs = []
    for s in steps:
        s.expect()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    for s in steps:
        s.q.mul_(0.5), s.bias.neg_(), s.lam[0].neg_()
    wants = [s.expect() for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for s, w in zip(steps, wants):
        s.check(w)


def test_captured_autograd():
    """A training step captured with leaves of its own."""
    S, D = 300, 64
    s = Step(S, D, torch.float16, 9)

    def step():
        leaves = [x.detach().requires_grad_(True) for x in (s.q, s.k, s.v, s.bias, *s.lam)]
        y = biased_attention(*leaves[:3], s.rp, s.ci, leaves[3], GEO)
        y = differential_attention(y, leaves[1], leaves[2], s.rp, s.ci, *leaves[4:], INIT)
        return [y.detach(), *torch.autograd.grad(y, leaves, s.do)]

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    torch.cuda.current_stream().wait_stream(st)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    s.v.mul_(-0.5)
    want = [x.clone() for x in step()]
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert tsa.tsa_last_device_status() == 0
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_calls_at_once_on_two_streams():
    steps = [Step(1000, 128, torch.bfloat16, 5), Step(900, 64, torch.float16, 6)]
    wants = [s.expect() for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(10):
        for s, st in zip(steps, streams):
            s.run(st)
    torch.cuda.synchronize()
    for s, w in zip(steps, wants):
        s.check(w)


def test_results_made_for_another_stream():
    """Outputs and workspaces that a call makes for a stream other than the current one outlive their
    last reference until that stream has used them."""
    s = Step(1000, 64, torch.float16, 8)
    o, lse = tsa.tsa_biased_attention_fwd(s.q, s.k, s.v, s.rp, s.ci, s.bias, GEO)
    args = (s.q, s.k, s.v, o, s.do, lse, s.rp, s.ci, s.bias, GEO)
    want = tsa.tsa_biased_attention_backward(*args)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        got = tsa.tsa_biased_attention_backward(*args, stream=st)
        rubbish = [torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV) for _ in range(8)]  # may reuse freed memory
        st.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        del rubbish
    assert tsa.tsa_last_device_status() == 0


def test_bucket_starts_are_read_by_the_forward():
    """A caller's list may change between the forward and the backward."""
    s = Step(300, 64, torch.float16, 10)
    want = s.expect()
    leaves = [x.requires_grad_(True) for x in (s.q, s.k, s.v, s.bias)]
    starts = list(GEO)
    y = biased_attention(*leaves[:3], s.rp, s.ci, leaves[3], starts)
    starts[1:] = [10 ** 6] * (len(starts) - 1)
    for x, w in zip(torch.autograd.grad(y, leaves, s.do), want[5:9]):
        assert torch.equal(x, w)


def test_strided_inputs_and_shared_biases():
    """[B, S, H, D] tensors seen as [B, H, S, D], and one bias row for all heads: its gradient is the sum."""
    B, H, S, D = 2, 3, 200, 64
    q, k, v, do = (_rand((B, H, S, D), torch.float16, 60 + i) for i in range(4))
    bias, lam = _learned(1, D, torch.float16, 61)
    rp, ci = _csr("dense", S, 64)
    leaves = [x.transpose(1, 2).contiguous().to(DEV).requires_grad_(True) for x in (q, k, v)]
    bd = bias.to(DEV).requires_grad_(True)
    y = biased_attention(*(x.transpose(1, 2) for x in leaves), *_dev(rp, ci), bd.expand(H, -1), GEO)
    grads = torch.autograd.grad(y, [*leaves, bd], do.transpose(1, 2).contiguous().to(DEV).transpose(1, 2))
    ref = biased(q, k, v, rp, ci, 64, D ** -0.5, bias.expand(H, -1), GEO, do)
    _close(y, *ref["O"], "O")
    for name, x in zip(BIASED, grads[:3]):
        _close(x.transpose(1, 2), *ref[name], name)
    val, err = ref["dbias"]
    val, err = val.sum(0, keepdim=True), err.sum(0, keepdim=True)
    # torch adds the heads' rounded rows and rounds the sum, in 16 bits at worst: H roundings
    _close(grads[3], val, err + H * U[torch.float16] * ref["dbias"][0].abs().sum(0, keepdim=True), "dbias")
    assert tsa.tsa_last_device_status() == 0


@pytest.mark.parametrize("S", [4096, 4097])
def test_backward_on_both_sides_of_the_short_schedule(S):
    """64 blocks: the transposed schedule is built by one launch; 65: by several."""
    B, H, D = 1, 1, 64
    q, k, v, do = (_rand((B, H, S, D), torch.float16, 70 + i) for i in range(4))
    bias, lam = _learned(H, D, torch.float16, 71)
    rp, ci = _csr("random", S, 64, 3)
    args = [x.to(DEV) for x in (q, k, v)]
    rpd, cid = _dev(rp, ci)
    dod, bd, ld = do.to(DEV), bias.to(DEV), [x.to(DEV) for x in lam]
    o, lse = tsa.tsa_biased_attention_fwd(*args, rpd, cid, bd, GEO)
    got = tsa.tsa_biased_attention_backward(*args, o, dod, lse, rpd, cid, bd, GEO)
    ref = biased(q, k, v, rp, ci, 64, D ** -0.5, bias, GEO, do)
    for name, x in zip(BIASED, got):
        _close(x, *ref[name], name)
    del ref
    o, o2, lse = tsa.tsa_differential_attention_fwd(*args, rpd, cid, *ld, INIT)
    got = tsa.tsa_differential_attention_backward(*args, o, o2, dod, lse, rpd, cid, *ld, INIT)
    ref = differential(q, k, v, rp, ci, 64, (D / 2) ** -0.5, lam, INIT, do)
    for name, x in zip(DIFF, got):
        _close(x, *ref[name], name)
    assert tsa.tsa_last_device_status() == 0


def _near_diagonal(nb):
    """Rows of the block before and the block itself."""
    ptr = np.concatenate([[0], 1 + 2 * np.arange(nb)])
    idx = np.stack([np.arange(nb) - 1, np.arange(nb)], 1).reshape(-1)[1:]
    return _dev(ptr, idx)


@pytest.mark.parametrize("which", ["biased", "differential"])
def test_offsets_past_32_bits(which):
    """Tensors of more than 2^31 elements: the last head is the same as when it runs alone."""
    H, S, D, dtype = 33, 64 * 8192 - 5, 128, torch.bfloat16
    assert H * S * D > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k, v, do = (torch.randn((1, H, S, D), dtype=dtype, generator=g, device=DEV) for _ in range(4))
    rp, ci = _near_diagonal(8192)
    bias, lam = _learned(H, D, dtype, 2)
    if which == "biased":
        extra = lambda h: (bias.to(DEV)[h:], GEO)  # noqa: E731
        fwd, bwd = tsa.tsa_biased_attention_fwd, tsa.tsa_biased_attention_backward
    else:
        extra = lambda h: (*(x.to(DEV) for x in lam), INIT)  # noqa: E731
        fwd, bwd = tsa.tsa_differential_attention_fwd, tsa.tsa_differential_attention_backward
    *outs, lse = fwd(q, k, v, rp, ci, *extra(0))
    grads = bwd(q, k, v, *outs, do, lse, rp, ci, *extra(0))
    got = [x[:, -1].clone() for x in (*outs, *grads[:3])]
    if which == "biased":
        got.append(grads[3][-1:].clone())
    del grads, outs, lse
    q, k, v, do = (x[:, -1:].contiguous() for x in (q, k, v, do))
    *outs, lse = fwd(q, k, v, rp, ci, *extra(H - 1))
    grads = bwd(q, k, v, *outs, do, lse, rp, ci, *extra(H - 1))
    assert tsa.tsa_last_device_status() == 0
    for x, y in zip(got, (*outs, *grads)):
        assert torch.equal(x.reshape(-1), y.reshape(-1))


def test_cache_past_32_bits():
    """A cache of more than 2^31 elements; only the listed blocks are read."""
    H, D, dtype = 2, 128, torch.float16
    cap = (1 << 23) + 40
    assert H * cap * D > 2 ** 31
    nb = -(-cap // 64)
    k, v = (torch.full((1, H, cap, D), float("nan"), dtype=dtype, device=DEV) for _ in range(2))
    row = [0, 77, nb // 2, nb - 3, nb - 2, nb - 1]
    small = []
    for x, seed in ((k, 1), (v, 2)):
        part = _rand((1, H, 6 * 64, D), dtype, seed)
        for i, j in enumerate(row):
            n = min(64, cap - j * 64)
            x[:, :, j * 64:j * 64 + n] = part[:, :, i * 64:i * 64 + n].to(DEV)
        small.append(part)
    q = _rand((1, H, D), dtype, 3)
    bias, lam = _learned(H, D, dtype, 4)
    lens, lists = torch.tensor([cap], dtype=torch.int32, device=DEV), _lists([row])
    one = tsa.tsa_biased_attention_decode(q.to(DEV), k, v, lens, *lists, bias.to(DEV), GEO)
    two = tsa.tsa_differential_attention_decode(q.to(DEV), k, v, lens, *lists, *(x.to(DEV) for x in lam), INIT)
    assert tsa.tsa_last_device_status() == 0
    few = 5 * 64 + 40  # the same keys gathered; the last block holds 40
    e1, e2 = (torch.exp((a.double() * b.double()).sum(-1)) for a, b in (lam[:2], lam[2:]))
    want, bound = _reference(q, *small, [few], [list(range(6))], 64, (D / 2) ** -0.5, lam=(e1 - e2 + INIT).expand(H))
    _close(two, want, bound, "differential")
    want, bound = _reference(q, *small, [few], [list(range(6))], 64, D ** -0.5, bias, GEO)
    # gathered, the first three blocks' keys lie far enough before the query for the last bucket, as in the cache
    assert few - 1 - 191 >= GEO[-1]
    _close(one, want, bound, "biased")


@pytest.mark.parametrize("which", ["biased", "differential"])
@pytest.mark.parametrize("D", [64, 128])
def test_wait_that_runs_out_is_reported(which, D):
    s = Step(700, D, torch.float16, 12)
    want = s.expect()
    call = (lambda: tsa.tsa_biased_attention(s.q, s.k, s.v, s.rp, s.ci, s.bias, GEO)) if which == "biased" else \
        (lambda: tsa.tsa_differential_attention(s.q, s.k, s.v, s.rp, s.ci, *s.lam, INIT))
    tsa.tsa_debug_set_wait_injection(True)
    try:
        call()
        assert tsa.tsa_last_device_status() == 7  # TSA_ERR_TIMEOUT
    finally:
        tsa.tsa_debug_set_wait_injection(False)
    assert torch.equal(call(), want[0 if which == "biased" else 1])
    s.run()
    s.check(want)


def test_refusals():
    s = Step(300, 64, torch.float16, 14)
    a, r = (s.q, s.k, s.v), (s.rp, s.ci)
    b16 = s.bias.to(torch.bfloat16)
    for bad in (lambda: tsa.tsa_biased_attention(*a, *r, b16, GEO), lambda: tsa.tsa_biased_attention(*a, *r, s.bias[:1], GEO),
                lambda: tsa.tsa_biased_attention(*a, *r, s.bias.cpu(), GEO),
                lambda: tsa.tsa_biased_attention(*a, *r, s.bias.t().contiguous().t(), GEO),
                lambda: tsa.tsa_biased_attention(*a, *r, s.bias, GEO[:-1]),
                lambda: tsa.tsa_biased_attention(*a, *r, s.bias, torch.tensor(GEO, device=DEV)),
                lambda: tsa.tsa_biased_attention(*a, s.rp[:-1], s.ci, s.bias, GEO),
                lambda: tsa.tsa_biased_attention(*a, s.rp.long(), s.ci, s.bias, GEO),
                lambda: tsa.tsa_biased_attention(*a, s.rp, s.ci.cpu(), s.bias, GEO),
                lambda: tsa.tsa_biased_attention(*a, *r, s.bias, GEO, out=s.o[:, :1]),
                lambda: tsa.tsa_biased_attention(s.q.transpose(1, 2), s.k, s.v, *r, s.bias, GEO),
                lambda: tsa.tsa_biased_attention(s.q.float(), s.k.float(), s.v.float(), *r, s.bias.float(), GEO),
                lambda: tsa.tsa_differential_attention(*a, *r, *s.lam[:3], s.lam[3][0], INIT),
                lambda: tsa.tsa_differential_attention(*a, *r, *(x.expand(3, -1).contiguous() for x in s.lam), INIT),
                lambda: tsa.tsa_differential_attention(*a, *r, *(x.float() for x in s.lam), INIT),
                lambda: tsa.tsa_biased_attention_backward(*a, s.o, s.do, s.lse2, *r, s.bias, GEO),
                lambda: tsa.tsa_biased_attention_backward(*a, s.o, s.do, s.lse, *r, s.bias, GEO, workspace=s.ws.float()),
                lambda: tsa.tsa_biased_attention_backward(*a, s.o, s.do, s.lse, *r, s.bias, GEO, dbias=s.bias[:1]),
                lambda: tsa.tsa_biased_attention_decode(s.last[0], s.k, s.v, s.lens, *s.lists, s.bias, GEO),
                lambda: tsa.tsa_biased_attention_decode(s.last, s.k[:, :1], s.v, s.lens, *s.lists, s.bias, GEO),
                lambda: tsa.tsa_biased_attention_decode(s.last, s.k, s.v, s.lens.long(), *s.lists, s.bias, GEO)):
        with pytest.raises((ValueError, TypeError)):
            bad()
    for bad, code in ((lambda: tsa.tsa_biased_attention(*a, *r, s.bias, GEO[::-1]), 1),
                      (lambda: tsa.tsa_biased_attention(*a, *r, s.bias, GEO, out=s.q), 1),
                      (lambda: tsa.tsa_biased_attention(*a, *r, s.bias, GEO, block=16), None),
                      (lambda: tsa.tsa_biased_attention(*a, *r, s.bias, GEO, scale=-1.0), 1),
                      (lambda: tsa.tsa_differential_attention(*a, *r, *s.lam, float("nan")), 1),
                      (lambda: tsa.tsa_biased_attention_backward(*a, s.o, s.do, s.lse, *r, s.bias, GEO, workspace=s.ws[:64]), 5),
                      (lambda: tsa.tsa_biased_attention_backward(*a, s.o, s.do, s.lse, *r, s.bias, GEO, dq=s.o), 1)):
        with pytest.raises((tsa.TsaError, ValueError)) as e:
            bad()
        if code is not None:
            assert e.value.status == code
    assert tsa.tsa_last_device_status() == 0
