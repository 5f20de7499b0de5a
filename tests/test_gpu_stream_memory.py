"""Outputs and workspaces that a call makes for a stream other than the current one: the current stream's
pending work writes nothing into them, and reads them whole after their last reference is gone."""
import pytest
import torch

import topology_scheduled_gb300 as tsa
from test_gpu_biased import DEV, STARTS, _csr, _dev
from test_gpu_decode import _lists

pytestmark = pytest.mark.gpu
GEO = STARTS["geometric"]
WAIT = 20_000_000  # clock ticks, some ten milliseconds


def _calls():
    H, S, D = 2, 1000, 64
    g = torch.Generator().manual_seed(1)
    q, k, v, do = (torch.randn((1, H, S, D), generator=g).half().to(DEV) for _ in range(4))
    bias = torch.randn((H, len(GEO)), generator=g).half().to(DEV)
    lam = [(0.2 * torch.randn((H, D // 2), generator=g)).half().to(DEV) for _ in range(4)]
    rp, ci = _dev(*_csr("random", S, 64, 1))
    last, lens, lists = q[:, :, -1].contiguous(), torch.tensor([S], dtype=torch.int32, device=DEV), _lists([list(range(16))])
    ob, lb = tsa.tsa_biased_attention_fwd(q, k, v, rp, ci, bias, GEO)
    op, lp = tsa.tsa_scheduled_attention_fwd(q, k, v, rp, ci)
    starts = torch.tensor([0, 130, 700], dtype=torch.int32, device=DEV)
    sums = tsa.tsa_block_sums(k)
    od, o2, ld = tsa.tsa_differential_attention_fwd(q, k, v, rp, ci, *lam, 0.5)
    return {
        "schedule": lambda s: tsa.tsa_build_schedule(k, salience=True, stream=s),
        "block sums": lambda s: (tsa.tsa_block_sums(k, stream=s),),
        "schedule from sums": lambda s: tsa.tsa_build_schedule_from_sums(sums, S=S, salience=True, stream=s),
        "segments": lambda s: tsa.tsa_segment_csr(960, 64, starts, stream=s),
        "fixed segments": lambda s: tsa.tsa_fixed_segment_csr(4096, 64, 512, stream=s),
        "dense": lambda s: tsa.tsa_dense_causal_csr(64000, stream=s),
        "plain": lambda s: tsa.tsa_scheduled_attention_fwd(q, k, v, rp, ci, stream=s),
        "plain backward": lambda s: tsa.tsa_scheduled_attention_backward(q, k, v, op, do, lp, rp, ci, stream=s),
        "biased": lambda s: tsa.tsa_biased_attention_fwd(q, k, v, rp, ci, bias, GEO, stream=s),
        "biased backward": lambda s: tsa.tsa_biased_attention_backward(q, k, v, ob, do, lb, rp, ci, bias, GEO, stream=s),
        "differential": lambda s: tsa.tsa_differential_attention_fwd(q, k, v, rp, ci, *lam, 0.5, stream=s),
        "differential backward": lambda s: tsa.tsa_differential_attention_backward(q, k, v, od, o2, do, ld, rp, ci, *lam, 0.5,
                                                                                   stream=s),
        "biased decode": lambda s: (tsa.tsa_biased_attention_decode(last, k, v, lens, *lists, bias, GEO, stream=s),),
        "differential decode": lambda s: (tsa.tsa_differential_attention_decode(last, k, v, lens, *lists, *lam, 0.5, stream=s),),
    }


def _written(which, x, results):
    """What of a result the call writes: the first row_ptr[-1] entries of a col_idx of that capacity."""
    if which in ("schedule", "schedule from sums", "segments") and x is results[1]:
        return x[:int(results[0][-1])]
    return x


@pytest.mark.parametrize("which", ["schedule", "block sums", "schedule from sums", "segments", "fixed segments", "dense",
                                   "plain", "plain backward", "biased", "biased backward", "differential",
                                   "differential backward", "biased decode", "differential decode"])
@pytest.mark.parametrize("raw", [False, True])
def test_memory_for_another_stream(which, raw):
    call = _calls()[which]
    want = [x.clone() for x in call(None)]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for _ in range(3):
        # memory of the results' sizes, still to be written by the current stream, and given back
        torch.cuda._sleep(WAIT)
        late = [torch.empty_like(x).fill_(7.0) for x in want for _ in range(3)]
        late += [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in (1 << 16, 1 << 18, 1 << 20, 1 << 21)]
        del late
        got = call(st.cuda_stream if raw else st)
        st.synchronize()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(_written(which, x, got), _written(which, y, want))
        # results read by the current stream after their last reference is gone
        torch.cuda._sleep(WAIT)
        copies = [x + 0 for x in got]
        del got, x
        call(st)
        more = []
        with torch.cuda.stream(st):
            more = [torch.empty_like(y).fill_(9.0) for y in want for _ in range(3)]
        torch.cuda.synchronize()
        for x, y in zip(copies, want):
            assert torch.equal(_written(which, x, copies), _written(which, y, want))
        del more
    assert tsa.tsa_last_device_status() == 0


def test_another_stream_within_a_capture():
    """Calls on a stream that forks from the captured one, their memory the graph's; replayed with other work
    between the replays."""
    calls = _calls()
    names = ["plain backward", "biased", "biased backward", "differential", "differential backward", "biased decode"]
    want = {n: [x.clone() for x in calls[n](None)] for n in names}
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.wait_stream(torch.cuda.current_stream())
        got = {n: calls[n](st) for n in names}
        torch.cuda.current_stream().wait_stream(st)
    for _ in range(3):
        for x in sum((list(v) for v in got.values()), []):
            x.fill_(7.0)
        g.replay()
        rubbish = [torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV) for _ in range(8)]
        torch.cuda.synchronize()
        for n in names:
            for x, y in zip(got[n], want[n]):
                assert torch.equal(x, y), n
        del rubbish
    assert tsa.tsa_last_device_status() == 0
