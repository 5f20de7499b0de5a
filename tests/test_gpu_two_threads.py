"""Calls of different lengths from several host threads at once."""
import threading

import pytest
import torch

import topology_scheduled_gb300 as tsa
from test_gpu_biased import DEV

pytestmark = pytest.mark.gpu


class Call:
    """A backward pass on a stream of its own, every tensor allocated beforehand."""

    def __init__(self, blocks, seed):
        S, D = 64 * blocks, 64
        g = torch.Generator(device=DEV).manual_seed(seed)
        q, k, v, do = (torch.randn((1, 1, S, D), dtype=torch.float16, generator=g, device=DEV) for _ in range(4))
        bias = torch.randn((1, 2), dtype=torch.float16, generator=g, device=DEV)
        rp = torch.arange(blocks + 1, dtype=torch.int32, device=DEV)
        ci = torch.arange(blocks, dtype=torch.int32, device=DEV)
        o, lse = tsa.tsa_biased_attention_fwd(q, k, v, rp, ci, bias, [0, 7])
        self.args = (q, k, v, o, do, lse, rp, ci, bias, [0, 7])
        self.out = dict(dq=torch.empty_like(q), dk=torch.empty_like(q), dv=torch.empty_like(q), dbias=torch.empty_like(bias))
        need = tsa.lib().tsa_biased_attention_backward_workspace_bytes(1, S, 64, blocks, 2)
        self.ws = torch.empty(need, dtype=torch.uint8, device=DEV)
        self.stream = torch.cuda.Stream()

    def __call__(self):
        tsa.tsa_biased_attention_backward(*self.args, **self.out, workspace=self.ws, stream=self.stream)


def test_lengths_do_not_disturb_each_other():
    """(4097 blocks are sorted in 64 KB of shared memory, 65 in 1 KB.)"""
    calls = [Call(4097, 1), Call(65, 2), Call(66, 5)]
    for c in calls:
        c()
    torch.cuda.synchronize()
    want = [{n: x.clone() for n, x in c.out.items()} for c in calls]
    errors, done = [], threading.Event()

    def loop(call, times):
        for i in range(times):
            if done.is_set():
                break
            try:
                call()
            except tsa.TsaError as e:
                errors.append(e)
            if i % 50 == 49:
                call.stream.synchronize()

    short = [threading.Thread(target=loop, args=(c, 10 ** 6)) for c in calls[1:]]
    for t in short:
        t.start()
    loop(calls[0], 2000)
    done.set()
    for t in short:
        t.join()
    torch.cuda.synchronize()
    assert tsa.tsa_last_device_status() == 0
    assert not errors, f"{len(errors)} calls refused, the first: {errors[0]}"
    for c, w in zip(calls, want):
        for n, x in c.out.items():
            assert torch.equal(x, w[n]), n


def test_builders_do_not_disturb_each_other():
    """(The graph phase of 4096 blocks takes 136 KB of shared memory, that of 64 blocks 12 KB.)"""
    def builder(blocks, seed):
        k = torch.randn((1, 64 * blocks, 64), dtype=torch.float16, generator=torch.Generator(device=DEV).manual_seed(seed),
                        device=DEV)
        ws = torch.empty(tsa.tsa_build_schedule_workspace_bytes(1, 64 * blocks, 64, 64), dtype=torch.uint8, device=DEV)
        rp = torch.empty(blocks + 1, dtype=torch.int32, device=DEV)
        ci = torch.zeros(tsa.tsa_schedule_max_nnz(64 * blocks, 64, 1, 1, 2), dtype=torch.int32, device=DEV)
        stream = torch.cuda.Stream()
        return (lambda: tsa.tsa_build_schedule(k, 64, 1, 1, 2, workspace=ws, row_ptr=rp, col_idx=ci, stream=stream)), rp, ci, stream

    builders = [builder(4096, 1), builder(64, 2), builder(65, 3)]
    for b in builders:
        b[0]()
    torch.cuda.synchronize()
    want = [(rp.clone(), ci.clone()) for _, rp, ci, _ in builders]
    errors, done = [], threading.Event()

    def loop(b, times):
        for i in range(times):
            if done.is_set():
                break
            try:
                b[0]()
            except tsa.TsaError as e:
                errors.append(e)
            if i % 20 == 19:
                b[3].synchronize()

    short = [threading.Thread(target=loop, args=(b, 10 ** 6)) for b in builders[1:]]
    for t in short:
        t.start()
    loop(builders[0], 1500)
    done.set()
    for t in short:
        t.join()
    torch.cuda.synchronize()
    assert tsa.tsa_last_device_status() == 0
    assert not errors, f"{len(errors)} calls refused, the first: {errors[0]}"
    for (_, rp, ci, _), (r, c) in zip(builders, want):
        assert torch.equal(rp, r) and torch.equal(ci, c)
