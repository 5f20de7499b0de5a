"""Rotary positions and the paged cache without a GPU: refusals, frequencies, and the 64-bit forms of the GPU tests."""
import math
import os
import re
from array import array

import pytest
import torch

import topology_scheduled_gb300 as tsa
from _cache import attention, gathered, page_lists, rotated
from topology_scheduled_gb300.binding import SIGNATURES

F = 1 << 20  # any aligned address: never read on these paths
M = 1 << 26  # farther apart than a tensor of the calls below is long
INVALID, UNSUPPORTED, CAPACITY = 1, 2, 5


def _passes(status):
    """The arguments are taken: what stops the call is that there is no device memory behind them."""
    return status in (3, 4, 6)


def _f(*values):
    return array("d", values or [1.0] * 32)


def _rotary(**change):
    f = _f()
    a = dict(Q=F, K=F + M, strides=None, positions=None, rows=1, frequencies=f.buffer_info()[0], R=64, interleaved=0,
             magnitude=1.0, inverse=0, Q_out=F + 2 * M, K_out=F + 3 * M, dtype=1, B=2, H=4, HK=2, S=100, D=64, stream=None)
    assert set(change) <= set(a)
    a.update(change)
    keep = [a["frequencies"], a["strides"]]
    for name in ("frequencies", "strides"):
        if isinstance(a[name], array):
            a[name] = a[name].buffer_info()[0]
    return tsa.lib().tsa_rotary(*a.values()) if keep else None


def _append(**change):
    f = _f()
    a = dict(Q=F, K=F + M, V=F + 2 * M, strides=None, K_cache=F + 3 * M, V_cache=F + 4 * M, pages=50, size=16, k_stride=2048,
             v_stride=2048, table=F + 5 * M, most=10, lens=F + 6 * M, counts=None, frequencies=f.buffer_info()[0], R=64,
             interleaved=0, magnitude=1.0, Q_out=F + 7 * M, dtype=1, B=2, H=4, HK=2, T=100, D=64, stream=None)
    assert set(change) <= set(a)
    a.update(change)
    keep = [a["frequencies"], a["strides"]]
    for name in ("frequencies", "strides"):
        if isinstance(a[name], array):
            a[name] = a[name].buffer_info()[0]
    return tsa.lib().tsa_paged_append(*a.values()) if keep else None


def _decode(**change):
    a = dict(Q=F, K_cache=F + M, V_cache=F + 2 * M, pages=50, size=16, k_stride=2048, v_stride=2048, table=F + 3 * M, most=10,
             lens=F + 4 * M, row_ptr=None, col_idx=None, nnz=0, O=F + 5 * M, dtype=1, B=2, H=4, HK=2, D=64, block=64,
             scale=0.125, ws=None, ws_bytes=0, stream=None)
    assert set(change) <= set(a)
    a.update(change)
    return tsa.lib().tsa_paged_attention_decode(*a.values())


def test_every_declared_symbol_is_exported_and_bound():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "tsa_cache.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(tsa_[a-z_0-9]+)\s*\(", text)))
    assert names == sorted(n for n in SIGNATURES if "rotary" in n or "paged" in n) and len(names) == 4
    for n in names:
        assert hasattr(tsa.lib(), n), n


def test_valid_calls_get_as_far_as_the_device():
    for status in (_rotary(), _rotary(K=None, K_out=None, HK=0), _append(), _append(Q=None, Q_out=None, H=0),
                   _append(Q=None, Q_out=None, frequencies=None, R=0), _decode(),
                   _decode(row_ptr=F + 6 * M, col_idx=F + 7 * M, nnz=9)):
        assert _passes(status), status


@pytest.mark.parametrize("change", [
    dict(Q=None), dict(Q_out=None), dict(K=None), dict(K_out=None), dict(frequencies=None), dict(dtype=2), dict(B=0), dict(S=0),
    dict(H=0), dict(HK=-1), dict(D=0), dict(R=0), dict(R=-16), dict(magnitude=float("nan")), dict(magnitude=float("inf")),
    dict(Q=F + 8), dict(K_out=F + 3 * M + 2), dict(positions=F + 5 * M + 2), dict(positions=F + 5 * M, rows=3),
    dict(positions=F + 5 * M, rows=0), dict(Q_out=F + 16), dict(Q_out=F + M), dict(K_out=F + 2 * M + 1024), dict(K_out=F),
    dict(positions=F + 2 * M + 64), dict(frequencies=_f(*[1.0] * 31, math.nan)), dict(frequencies=_f(*[1.0] * 31, 65537.0))])
def test_rotary_arguments(change):
    assert _rotary(**change) == INVALID, change


@pytest.mark.parametrize("change", [dict(R=24), dict(R=80), dict(D=72, R=16), dict(D=272), dict(H=65536), dict(B=1 << 16, S=1 << 16),
                                    dict(S=1 << 31)])
def test_rotary_sizes(change):
    assert _rotary(**change) == UNSUPPORTED, change


def _joint(S=100, heads=8, D=64, q=4, k=2):
    """Strides of Q and K as heads of one projection [B, S, heads, D], and K's place behind Q."""
    one = (S * heads * D, D, heads * D)
    return one, q * D * 2


def test_rows_of_one_array():
    """Outputs may lie between the rows of another tensor, not on them."""
    one, behind = _joint()
    four = array("q", one * 4)
    # Q and K in place, side by side in one projection
    assert _passes(_rotary(strides=four, K=F + behind, Q_out=F, K_out=F + behind))
    # K's heads begin on Q's last one
    assert _rotary(strides=four, K=F + behind - 128, Q_out=F, K_out=F + behind - 128) == INVALID
    # in place, with other strides
    assert _rotary(strides=array("q", one * 2 + (4 * 6400, 6400, 64) + one), K=F + behind, Q_out=F, K_out=F + behind) == INVALID
    # K_out wraps round a token's end onto the next one's Q
    assert _rotary(strides=four, K=F + behind, Q_out=F, K_out=F + 7 * 128) == INVALID
    # a stride that is no multiple of the other's period
    odd = (100 * 512 + 8, 64, 512)
    assert _rotary(strides=array("q", odd * 4), K=F + behind, Q_out=F, K_out=F + behind) == INVALID


def test_strides():
    dense = (4 * 6400, 6400, 64)
    k = (2 * 6400, 6400, 64)
    assert _passes(_rotary(strides=array("q", dense + k + dense + k)))
    for at, value in ((0, -8), (1, 4), (2, 63), (6, 0), (7, 0), (8, 56), (8, 1 << 60), (3, 1 << 59)):
        s = array("q", dense + k + dense + k)
        s[at] = value
        assert _rotary(strides=s) == INVALID, (at, value)
    s = array("q", (0, 0, 0) + (0, 0, 0) + dense + k)  # inputs may be broadcast
    assert _passes(_rotary(strides=s))
    s = array("q", dense + (-1, -1, -1) + dense + (-1, -1, -1))  # nor is a missing tensor's read
    assert _passes(_rotary(strides=s, K=None, K_out=None))
    s = array("q", (-3, 7, 5) * 4)  # an axis of one has no stride
    assert _passes(_rotary(strides=s, B=1, H=1, HK=1, S=1))


@pytest.mark.parametrize("change", [
    dict(K=None), dict(V=None), dict(K_cache=None), dict(V_cache=None), dict(table=None), dict(lens=None), dict(Q=None),
    dict(Q_out=None), dict(frequencies=None), dict(dtype=-1), dict(B=0), dict(T=0), dict(HK=0), dict(pages=0), dict(most=0),
    dict(size=0), dict(size=-16), dict(k_stride=2040), dict(k_stride=2052), dict(v_stride=0), dict(K_cache=F + 3 * M + 8),
    dict(V=F + 2 * M + 4), dict(lens=F + 6 * M + 1), dict(counts=F + 6 * M + 66), dict(Q_out=F + 32), dict(Q_out=F + 3 * M),
    dict(K_cache=F), dict(V_cache=F + 3 * M), dict(V_cache=F + M), dict(table=F + 3 * M), dict(lens=F + 7 * M),
    dict(counts=F + 4 * M), dict(magnitude=math.inf)])
def test_append_arguments(change):
    assert _append(**change) == INVALID, change


@pytest.mark.parametrize("change", [dict(size=8), dict(size=48), dict(size=512), dict(most=1 << 27), dict(pages=1 << 31), dict(R=40),
                                    dict(D=24), dict(HK=70000), dict(T=1 << 31)])
def test_append_sizes(change):
    assert _append(**change) == UNSUPPORTED, change


def test_caches_of_one_array():
    """[pages, 2, HK, page_size, D]: keys and values of a page side by side."""
    two = dict(k_stride=4096, v_stride=4096)
    assert _passes(_append(K_cache=F + 3 * M, V_cache=F + 3 * M + 4096, **two))
    assert _append(K_cache=F + 3 * M, V_cache=F + 3 * M + 4080, **two) == INVALID
    assert _append(K_cache=F + 3 * M, V_cache=F + 3 * M + 4112, **two) == INVALID
    assert _append(K_cache=F + 3 * M, V_cache=F + 3 * M + 4096, k_stride=4096, v_stride=8192) == INVALID
    assert _passes(_append(pages=1, k_stride=0, v_stride=-5))  # one page has no stride


@pytest.mark.parametrize("change", [
    dict(Q=None), dict(K_cache=None), dict(V_cache=None), dict(table=None), dict(lens=None), dict(O=None), dict(row_ptr=F),
    dict(col_idx=F), dict(nnz=4), dict(row_ptr=F + 6 * M, col_idx=F + 7 * M, nnz=0), dict(nnz=-1), dict(dtype=7), dict(B=0),
    dict(H=0), dict(HK=0), dict(HK=3), dict(D=0), dict(block=0), dict(scale=0.0), dict(scale=math.nan), dict(scale=-1.0),
    dict(Q=F + 2), dict(O=F + 5 * M + 8), dict(lens=F + 2), dict(ws=F + 128), dict(O=F), dict(O=F + M + 512),
    dict(O=F + 4 * M), dict(row_ptr=F + 5 * M, col_idx=F + 7 * M, nnz=9), dict(k_stride=100)])
def test_decode_arguments(change):
    assert _decode(**change) == INVALID, change


@pytest.mark.parametrize("change", [dict(D=96), dict(D=256), dict(block=16), dict(size=8), dict(size=24), dict(size=512),
                                    dict(B=1 << 16), dict(H=1 << 16, HK=1), dict(most=1 << 27), dict(pages=1 << 32),
                                    dict(row_ptr=F + 6 * M, col_idx=F + 7 * M, nnz=1 << 30)])
def test_decode_sizes(change):
    assert _decode(**change) == UNSUPPORTED, change


def test_decode_workspace():
    need = tsa.tsa_paged_attention_decode_workspace_bytes
    long = dict(B=1, H=1, HK=1, D=64, size=64, most=1000, k_stride=4096, v_stride=4096)
    bytes_ = need(1, 1, 1, 64, 64, 1000)
    assert bytes_ > 0 and need(64, 32, 32, 128, 64, 1000) == 0 and need(1, 1, 1, 64, 64, 1) == 0
    assert _decode(**long) == INVALID  # none given
    assert _decode(**long, ws=F + 6 * M, ws_bytes=bytes_ - 1) == CAPACITY
    assert _passes(_decode(**long, ws=F + 6 * M, ws_bytes=bytes_))
    assert _decode(**long, ws=F + M, ws_bytes=bytes_) == INVALID  # on the cache
    assert _decode(**long, ws=F + 5 * M, ws_bytes=bytes_) == INVALID  # on the output
    for bad in ((0, 1, 1, 64, 64, 10), (1, 3, 2, 64, 64, 10), (1, 1, 1, 96, 64, 10), (1, 1, 1, 64, 8, 10), (1, 1, 1, 64, 64, 0),
                (1, 1, 1, 64, 64, 10, 16), (1, 1, 1, 64, 64, 10, 64, -1), (1 << 40, 1, 1, 64, 64, 10)):
        assert need(*bad) == 0, bad
    # any split's parts fit: no size overflows
    assert need(1, 32, 8, 128, 64, 1 << 24) < 1 << 30


def test_binding_checks_need_no_gpu():
    x = torch.zeros((1, 1, 4, 64), dtype=torch.float16)
    f = tsa.rotary_frequencies(64)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        tsa.tsa_rotary(x, x, f)
    with pytest.raises(ValueError):
        tsa.tsa_paged_append(None, x, x, x, x, i[None], i)
    with pytest.raises(ValueError):
        tsa.tsa_paged_attention_decode(x[0], x, x, i[None], i)


def test_frequencies():
    f = tsa.rotary_frequencies(8, 10000.0)
    assert list(f) == [10000.0 ** (-i / 4) for i in range(4)] and f.typecode == "d"
    assert list(tsa.rotary_frequencies(8, 10000.0, scaling="linear", factor=4.0)) == [x / 4 for x in f]
    # a larger base: the first pair as it is, the last one divided by the factor
    g = tsa.rotary_frequencies(8, 10000.0, scaling="base", factor=4.0)
    assert g[0] == f[0] and math.isclose(g[3], f[3] / 4, rel_tol=1e-12)
    # a ramp: pairs that turn over 32 times in 8192 tokens stay, those under once are divided, none is out of order
    f = tsa.rotary_frequencies(128)
    g = tsa.rotary_frequencies(128, scaling="ramp", factor=4.0, original_length=8192)
    turns = [8192 * x / (2 * math.pi) for x in f]
    for x, y, t in zip(f, g, turns):
        if t >= 32:
            assert y == x
        elif t <= 1:
            assert math.isclose(y, x / 4, rel_tol=1e-12)
        else:
            assert x / 4 < y < x
            k = (t - 1) / 31
            assert math.isclose(y, x * k + x / 4 * (1 - k), rel_tol=1e-12)
    assert all(a > b for a, b in zip(g, list(g)[1:]))
    assert tsa.rotary_magnitude(1.0) == 1.0 and math.isclose(tsa.rotary_magnitude(4.0), 1 + 0.1 * math.log(4))
    for bad in (dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=8, base=0.0), dict(rotary_dim=8, factor=-1.0),
                dict(rotary_dim=8, scaling="other"), dict(rotary_dim=8, scaling="ramp", factor=2.0),
                dict(rotary_dim=8, scaling="ramp", factor=2.0, original_length=100, low=3.0, high=2.0),
                dict(rotary_dim=8, factor=math.inf)):
        with pytest.raises(ValueError):
            tsa.rotary_frequencies(**bad)


@pytest.mark.parametrize("interleaved", [False, True])
def test_form_of_the_rotation(interleaved):
    """Against complex numbers; rotations add up, and scores depend on distances alone."""
    g = torch.Generator().manual_seed(1)
    q, k = (torch.randn((1, 64), generator=g, dtype=torch.float64) for _ in range(2))
    f = [0.5 ** i for i in range(24)]  # 48 of 64 dimensions
    y, _ = rotated(q, [13], f, interleaved, 1.5)
    re, im = (q[0, 0:48:2], q[0, 1:48:2]) if interleaved else (q[0, :24], q[0, 24:48])
    z = 1.5 * torch.complex(re, im) * torch.polar(torch.ones(24, dtype=torch.float64), 13.0 * torch.tensor(f, dtype=torch.float64))
    want = torch.cat([torch.stack([z.real, z.imag], 1).flatten() if interleaved else torch.cat([z.real, z.imag]), q[0, 48:]])
    assert torch.allclose(y[0], want, rtol=0, atol=1e-13)
    there, _ = rotated(q, [13], f, interleaved)
    twice, _ = rotated(there, [29], f, interleaved)
    once, _ = rotated(q, [42], f, interleaved)
    assert torch.allclose(twice, once, rtol=0, atol=1e-13)
    back, _ = rotated(there, [13], f, interleaved, inverse=True)
    assert torch.allclose(back, q, rtol=0, atol=1e-13)
    near = float((rotated(q, [7], f, interleaved)[0] * rotated(k, [5], f, interleaved)[0]).sum())
    far = float((rotated(q, [(1 << 30) + 2], f, interleaved)[0] * rotated(k, [1 << 30], f, interleaved)[0]).sum())
    assert abs(near - far) < 1e-12


def test_form_of_the_attention():
    """One query over a cache is the last row of causal attention with every head's keys written out."""
    g = torch.Generator().manual_seed(2)
    K, V = (torch.randn((2, 37, 64), generator=g, dtype=torch.float64) for _ in range(2))
    q = torch.randn((6, 64), generator=g, dtype=torch.float64)
    O, bound = attention(q, K, V, 3, 0.125, torch.float16)
    for h in range(6):
        want = torch.nn.functional.scaled_dot_product_attention(q[None, h:h + 1], K[None, h // 3], V[None, h // 3], scale=0.125)
        assert torch.allclose(O[h], want[0, 0], rtol=0, atol=1e-14)
    assert bool((bound > 0).all()) and float(bound.max()) < 2e-3
    empty, none = attention(q, K[:, :0], V[:, :0], 3, 0.125, torch.float16)
    assert bool((empty == 0).all()) and bool((none == 0).all())


def test_form_of_the_pages():
    table, pages = page_lists([20, 0, 33], 16, seed=3)
    assert table.shape == (3, 3) and pages == 8
    used = table[table >= 0].tolist()
    assert len(used) == 5 == len(set(used)) and (table[1] == -1).all()
    cache = torch.arange(pages * 16).reshape(pages, 1, 16, 1).float()
    rows = gathered(cache, table[2], 33)
    assert [int(x) for x in rows.flatten()] == [int(table[2, k // 16]) * 16 + k % 16 for k in range(33)]
