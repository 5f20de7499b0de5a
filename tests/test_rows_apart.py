"""Rows of one array that share no memory may be rotated and appended in place, whichever axis keeps them apart; rows that
share some are refused.  (No GPU: a call that is taken ends where its memory is no device's.)"""
import random
from array import array

import pytest

import topology_scheduled_gb300 as tsa

F = 1 << 20  # any aligned address: never read on these paths
FAR = 1 << 30
INVALID, TAKEN = 1, (3, 4, 6)


def _rotary(B, S, H, HK, D, q, k, behind):
    """Q and K rotated in place, K `behind` elements behind Q."""
    f, strides = array("d", [1.0] * (D // 2)), array("q", (*q, *k) * 2)
    status = tsa.lib().tsa_rotary(F, F + 2 * behind, strides.buffer_info()[0], None, 1, f.buffer_info()[0], D, 0, 1.0, 0, F,
                                  F + 2 * behind, 1, B, H, HK, S, D, None)
    assert status == INVALID or status in TAKEN
    return status in TAKEN


def _append(B, T, H, HK, D, strides, q, k, v):
    """Q rotated in place beside the K and V that are appended."""
    f, s = array("d", [1.0] * (D // 2)), array("q", strides * 4)
    status = tsa.lib().tsa_paged_append(F + 2 * q, F + 2 * k, F + 2 * v, s.buffer_info()[0], F + FAR, F + 2 * FAR, 50, 16,
                                        HK * 16 * D, HK * 16 * D, F + 3 * FAR, 10, F + 4 * FAR, None, f.buffer_info()[0], D, 0,
                                        1.0, F + 2 * q, 1, B, H, HK, T, D, None)
    assert status == INVALID or status in TAKEN
    return status in TAKEN


@pytest.mark.parametrize("B,S", [(1, 1), (1, 100), (3, 1), (3, 100)])
def test_heads_first(B, S):
    """[B, H + 2 HK, S, D]."""
    H, HK, D = 4, 2, 64
    strides = ((H + 2 * HK) * S * D, S * D, D)
    assert _rotary(B, S, H, HK, D, strides, strides, H * S * D)
    assert _append(B, S, H, HK, D, strides, 0, H * S * D, (H + HK) * S * D)
    # K's first head is Q's last one; V's is the next batch's first of Q
    assert not _rotary(B, S, H, HK, D, strides, strides, (H - 1) * S * D)
    assert not _append(B, S, H, HK, D, strides, 0, (H - 1) * S * D, (H + HK) * S * D)
    assert _append(B, S, H, HK, D, strides, 0, H * S * D, (H + 2 * HK - 1) * S * D) == (B == 1)


@pytest.mark.parametrize("B,S", [(1, 1), (1, 100), (3, 1), (3, 100)])
def test_each_heads_together(B, S):
    """[B, S, H, 3, D]."""
    H, D = 4, 64
    strides = (S * H * 3 * D, 3 * D, H * 3 * D)
    assert _rotary(B, S, H, H, D, strides, strides, D)
    assert _append(B, S, H, H, D, strides, 0, D, 2 * D)
    assert not _rotary(B, S, H, H, D, strides, strides, D - 8)
    assert not _rotary(B, S, H, H, D, strides, strides, 3 * D)
    assert not _append(B, S, H, H, D, strides, 0, D, 2 * D + 8)


def test_rows_of_any_strides():
    """Against sets of elements: no call is taken whose rows meet, and every one whose rows lie one within another's gaps."""
    rng = random.Random(7)
    taken = refused = 0
    for _ in range(4000):
        B, S, H, HK, D = rng.randint(1, 3), rng.randint(1, 4), rng.randint(1, 3), rng.randint(1, 3), 16
        axes = rng.sample(range(3), 3)  # from the innermost outwards
        strides, at, n = [0, 0, 0], rng.choice([16, 24, 32, 48]), (B, max(H, HK), S)
        nested = rng.random() < 0.7
        for axis in axes:
            strides[axis] = at
            at = at * max(n[axis], 1) * rng.choice([1, 1, 2]) if nested else at + rng.choice([0, 8, 16, 32, 64])
        k = strides if rng.random() < 0.9 else [s + rng.choice([0, 8]) for s in strides]
        behind = 8 * rng.randint(-20, 80)

        def elements(first, st, heads):
            return {first + b * st[0] + h * st[1] + s * st[2] + d for b in range(B) for h in range(heads) for s in range(S) for d in range(D)}

        q_rows, k_rows = elements(0, strides, H), elements(behind, k, HK)
        whole = len(q_rows) == B * H * S * D and len(k_rows) == B * HK * S * D
        got = _rotary(B, S, H, HK, D, strides, k, behind)
        if got:
            assert whole and not q_rows & k_rows, (B, S, H, HK, strides, k, behind)
        elif nested and k is strides and whole:
            assert q_rows & k_rows, (B, S, H, HK, strides, behind)
        taken += got
        refused += not got
    assert taken > 500 and refused > 500


@pytest.mark.parametrize("B,S", [(1, 1), (1, 100), (3, 1), (3, 100)])
def test_heads_of_other_strides(B, S):
    """[B, S, 4 x 64 + 2 x 128]: Q's heads are 64 elements apart, K's 128, of which the first 64 are rotated."""
    H, HK, D, token = 4, 2, 64, 512
    q, k = (S * token, D, token), (S * token, 2 * D, token)
    if S > 1 or B > 1:
        assert _rotary(B, S, H, HK, D, q, k, H * D)
    assert not _rotary(B, S, H, HK, D, q, k, H * D - 8)
    assert not _rotary(B, S, H, HK, D, q, k, token + D) or (B, S) == (1, 1)
