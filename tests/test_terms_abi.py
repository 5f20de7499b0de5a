"""Refusals of the attentions with learned score terms that need no GPU, and their bucket starts."""
import ctypes
import os
import re

import pytest
import torch

import topology_scheduled_gb300 as tsa
from topology_scheduled_gb300.binding import SIGNATURES

F = 1 << 20        # any aligned address: never read on these paths
M = 1 << 24        # farther apart than a tensor of the calls below is long


def _starts(*values):
    return (ctypes.c_int32 * max(1, len(values)))(*values)


def _biased(**change):
    a = dict(Q=F, K=F + M, V=F + 2 * M, row_ptr=F, col_idx=F, nnz_cap=10, bias=F + 3 * M, starts=_starts(0, 1, 2, 8), n=4,
             O=F + 4 * M, lse=F + 5 * M, dtype=1, B=1, H=2, S=1024, D=64, block=64, scale=0.125, stream=None)
    a.update(change)
    return tsa.lib().tsa_biased_attention_fwd(*a.values())


def _diff(**change):
    a = dict(Q=F, K=F + M, V=F + 2 * M, row_ptr=F, col_idx=F, nnz_cap=10, lq1=F + 3 * M, lk1=F + 3 * M + 512,
             lq2=F + 3 * M + 1024, lk2=F + 3 * M + 1536, heads=2, init=0.5, O=F + 4 * M, O2=F + 5 * M, lse=F + 6 * M,
             dtype=1, B=1, H=2, S=1024, D=64, block=64, scale=0.125, stream=None)
    a.update(change)
    return tsa.lib().tsa_differential_attention_fwd(*a.values())


BOTH = [dict(Q=None), dict(row_ptr=None), dict(O=None), dict(dtype=7), dict(B=0), dict(S=0), dict(nnz_cap=0),
        dict(scale=0.0), dict(scale=-0.1), dict(scale=float("nan")), dict(Q=F + 8), dict(O=F + 4 * M + 2),
        dict(lse=F + 5 * M + 2), dict(O=F), dict(lse=F + M + 64), dict(row_ptr=F + 2)]


def test_every_declared_symbol_is_exported_and_bound():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "tsa_terms.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(tsa_[a-z_0-9]+)\s*\(", text)))
    assert names == sorted(n for n in SIGNATURES if "biased" in n or "differential" in n)
    for n in names:
        assert hasattr(tsa.lib(), n), n


@pytest.mark.parametrize("change", BOTH + [dict(bias=None), dict(starts=None), dict(n=0), dict(starts=_starts(1, 2, 3, 4)),
                                           dict(starts=_starts(0, 5, 4, 8)), dict(bias=F + 3 * M + 1),
                                           dict(lse=F + 4 * M)])
def test_biased_arguments(change):
    assert _biased(**change) == 1  # TSA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("change", BOTH + [dict(lq1=None), dict(lk2=None), dict(heads=3), dict(heads=0),
                                           dict(init=float("inf")), dict(lk1=F + 3), dict(O2=F + 4 * M),
                                           dict(O2=F + 5 * M + 4)])
def test_differential_arguments(change):
    assert _diff(**change) == 1


@pytest.mark.parametrize("change", [dict(D=96), dict(block=16), dict(H=70000), dict(S=1 << 31), dict(B=64, S=1 << 25),
                                    dict(nnz_cap=1 << 30)])
def test_sizes_that_are_not_supported(change):
    assert _biased(**change) == 2 and _diff(**change) == 2


def test_too_many_buckets():
    assert _biased(n=257, starts=_starts(*range(257))) == 2


def test_bucket_starts():
    s = tsa.relative_bucket_starts(32, 128)
    assert s[:17] == list(range(17)) and len(s) == 32 and s[-1] < 128
    for i in range(16):  # the border of bucket 16 + i, written out: 16 * 8 ** (i / 16)
        d = s[16 + i]
        assert d ** 16 >= 16 ** 16 * 8 ** i and (d - 1) ** 16 < 16 ** 16 * 8 ** i
    assert tsa.relative_bucket_starts(2, 2) == [0, 1]
    for n, most in ((0, 5), (3, 9), (258, 1000), (32, 16)):
        with pytest.raises(ValueError):
            tsa.relative_bucket_starts(n, most)


def test_binding_checks_need_no_gpu():
    x = torch.zeros((1, 1, 64, 64), dtype=torch.float16)
    rp, ci = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        tsa.tsa_biased_attention(x, x, x, rp, ci, torch.zeros((1, 2), dtype=torch.float16), [0, 1])
    with pytest.raises(ValueError):
        tsa.tsa_differential_attention(x, x, x, rp, ci, *(torch.zeros(32, dtype=torch.float16) for _ in range(4)), 0.5)


def _decode(which, **change):
    a = dict(Q=F, K=F + M, V=F + 2 * M, lens=F, row_ptr=F, col_idx=F, nnz_cap=10)
    a.update(dict(bias=F + 3 * M, starts=_starts(0, 1, 2, 8), n=4) if which == "biased" else
             dict(lq1=F + 3 * M, lk1=F + 3 * M + 512, lq2=F + 3 * M + 1024, lk2=F + 3 * M + 1536, heads=2, init=0.5))
    a.update(O=F + 4 * M, dtype=1, B=1, H=2, capacity=1024, D=64, block=64, scale=0.125, stream=None)
    assert set(change) <= set(a)
    a.update(change)
    return getattr(tsa.lib(), f"tsa_{which}_attention_decode")(*a.values())


@pytest.mark.parametrize("which", ["biased", "differential"])
def test_decode_arguments(which):
    for change in (dict(Q=None), dict(lens=None), dict(col_idx=None), dict(O=None), dict(B=0), dict(H=0), dict(capacity=0),
                   dict(D=0), dict(nnz_cap=0), dict(scale=0.0), dict(dtype=3), dict(Q=F + 8), dict(lens=F + 2), dict(O=F),
                   dict(O=F + M + 1024), dict(O=F + 3 * M)):
        assert _decode(which, **change) == 1, change
    for change in (dict(D=96), dict(block=16), dict(B=70000), dict(H=70000), dict(capacity=(1 << 31) - 1)):
        assert _decode(which, **change) == 2, change


def _back(which, **change):
    a = dict(Q=F, K=F + M, V=F + 2 * M, O=F + 3 * M)
    if which == "differential":
        a.update(O2=F + 4 * M)
    a.update(dO=F + 5 * M, lse=F + 6 * M, row_ptr=F, col_idx=F, nnz_cap=10)
    a.update(dict(bias=F + 7 * M, starts=_starts(0, 1, 2, 8), n=4) if which == "biased" else
             dict(lq1=F + 7 * M, lk1=F + 7 * M + 512, lq2=F + 7 * M + 1024, lk2=F + 7 * M + 1536, heads=2, init=0.5))
    a.update(dQ=F + 8 * M, dK=F + 9 * M, dV=F + 10 * M)
    a.update(dict(dbias=F + 11 * M) if which == "biased" else
             dict(d1=F + 11 * M, d2=F + 11 * M + 512, d3=F + 11 * M + 1024, d4=F + 11 * M + 1536))
    a.update(dtype=1, B=1, H=2, S=1024, D=64, block=64, scale=0.125, ws=F + 12 * M, ws_bytes=1 << 24, stream=None)
    assert set(change) <= set(a)
    a.update(change)
    return getattr(tsa.lib(), f"tsa_{which}_attention_backward")(*a.values())


@pytest.mark.parametrize("which", ["biased", "differential"])
def test_backward_arguments(which):
    first = "dbias" if which == "biased" else "d1"
    for change in (dict(O=None), dict(dO=None), dict(lse=None), dict(dV=None), dict(ws=None), {first: None}, dict(dQ=F),
                   dict(dK=F + 8 * M + 16), dict(dV=F + 5 * M), {first: F + 7 * M}, {first: F + 10 * M}, dict(ws=F + 12 * M + 8),
                   dict(ws=F + 9 * M), dict(dO=F + 5 * M + 8), dict(S=0), dict(scale=-1.0), {first: F + 11 * M + 1}):
        assert _back(which, **change) == 1, change
    for change in (dict(block=32), dict(D=96), dict(S=64 * 8193, nnz_cap=10), dict(B=64, H=64, S=1 << 19)):
        assert _back(which, **change) == 2, change
    assert _back(which, ws_bytes=1000) == 5


def test_workspace_bytes():
    L = tsa.lib()
    both = (lambda *a: L.tsa_biased_attention_backward_workspace_bytes(*a, 32),
            L.tsa_differential_attention_backward_workspace_bytes)
    for f in both:
        assert f(64, 32768, 64, 7000) > 64 * 32768 * 4 and f(1, 1, 128, 1) > 0
        for bad in ((0, 64, 64, 1), (70000, 64, 64, 1), (1, 0, 64, 1), (1, 64, 32, 1), (1, 64 * 8193, 64, 1), (1, 64, 64, 0),
                    (1 << 40, 1 << 30, 64, 1), (1, 1 << 40, 64, 1), (65535, 1 << 16, 64, 1)):
            assert f(*bad) == 0
    assert L.tsa_biased_attention_backward_workspace_bytes(1, 64, 64, 1, 257) == 0


@pytest.mark.parametrize("which", ["biased", "differential"])
def test_outputs_keep_off_the_schedule(which):
    """(The arrays of a schedule are inputs like any other.)"""
    at = F + 40 * M
    first = _biased if which == "biased" else _diff
    assert first(O=at, row_ptr=at) == 1 and first(O=at, col_idx=at + 16) == 1
    for change in (dict(dQ=at, row_ptr=at + 4), dict(ws=at, col_idx=at + 64), dict(dV=at, col_idx=at)):
        assert _back(which, **change) == 1, change
    for change in (dict(O=at, row_ptr=at), dict(O=at, lens=at + 4), dict(O=at, col_idx=at)):
        assert _decode(which, **change) == 1, change
