"""Rotary positions, the paged key/value cache and its one-token attention (include/tsa_cache.h).

``tsa_rotary``                 -- rotates the pairs of Q's and K's rows by their positions (or back);
``tsa_paged_append``           -- writes new tokens to a paged cache, rotating on the way;
``tsa_paged_attention_decode`` -- one new token per sequence against a paged cache.

Like the calls of ``binding`` they run in libtsa.so on the current stream (or ``stream``) and
raise when a call fails; there is no fallback. Their arguments are checked and marshalled in
csrc/calls.cpp: single tokens are too short for the interpreter. They have no gradients
(``autograd.rotary`` has): a tensor that they write in place may require none while gradients
are recorded, and counts as changed where autograd has kept it for a backward pass.
"""
from __future__ import annotations

import math
from array import array

import torch

from .binding import _on, calls, lib


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                       original_length: int | None = None, low: float = 1.0, high: float = 32.0) -> array:
    """The angle per position of each of the rotary_dim / 2 pairs, base ** (-2 i / rotary_dim), in 64 bits.

    ``scaling`` for contexts ``factor`` times as long as the ``original_length`` tokens trained on:
    ``"linear"`` divides every frequency by factor; ``"base"`` enlarges the base to
    base * factor ** (rotary_dim / (rotary_dim - 2)), which divides the last pair's by factor and leaves the
    first pair's; ``"ramp"`` divides the pairs that turn less than ``low`` times in original_length tokens,
    leaves those that turn more than ``high`` times, and blends between, linearly in the number of turns (its
    attention is sharpened by ``rotary_magnitude``). A model trained with another blend, such as one that is
    linear in the pair's number, is given its own frequencies: the calls take any."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and positive")
    if not base > 0 or not factor > 0 or not math.isfinite(base) or not math.isfinite(factor):
        raise ValueError("base and factor must be positive")
    if scaling not in (None, "linear", "base", "ramp"):
        raise ValueError(f"scaling must be None, 'linear', 'base' or 'ramp', got {scaling!r}")
    if scaling == "base" and rotary_dim > 2:
        base *= factor ** (rotary_dim / (rotary_dim - 2))
    f = [base ** (-2 * i / rotary_dim) for i in range(rotary_dim // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "ramp":
        if original_length is None or original_length <= 0 or not low < high:
            raise ValueError("scaling 'ramp' needs a positive original_length, and low below high")
        keep = [min(max((original_length * x / (2 * math.pi) - low) / (high - low), 0.0), 1.0) for x in f]
        f = [x * (k + (1 - k) / factor) for x, k in zip(f, keep)]
    return array("d", f)


def rotary_magnitude(factor: float) -> float:
    """Magnitude of rotated rows that goes with ``scaling="ramp"``: 0.1 ln(factor) + 1, and 1 up to factor 1."""
    return 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0


def _frequencies(frequencies):
    """The frequencies as a host array of binary64 (the library checks their values)."""
    if isinstance(frequencies, array) and frequencies.typecode == "d":
        return frequencies
    if isinstance(frequencies, torch.Tensor):
        if frequencies.is_cuda:
            raise ValueError("frequencies must be host numbers")
        frequencies = frequencies.tolist()
    return array("d", frequencies)


def _called(call, stream, like, given, args):
    """call(*args) on `stream`.  What it makes is then that stream's own memory, and is not given away before the
    current stream has done what it is asked to do with it; `given` outputs are left to the caller."""
    _, other = _on(stream, like.device)
    if other is None:
        return call(*args)
    here = torch.cuda.current_stream(like.device)
    with torch.cuda.stream(other):
        made = call(*args)
    for t, g in zip(made if isinstance(made, tuple) else (made,), given):
        if t is not None and g is None:
            t.record_stream(here)
    return made


def tsa_rotary(Q, K, frequencies, positions=None, *, interleaved: bool = False, magnitude: float = 1.0,
               inverse: bool = False, out=None, out_k=None, stream=None):
    """Rotary positions: every pair of the first 2 len(frequencies) dimensions of the rows of Q [B, H, S, D] and
    K [B, HK, S, D] is rotated by position * frequency and scaled by ``magnitude``; the rest is copied.  The
    pairs are (i, i + R/2), or (2 i, 2 i + 1) if ``interleaved``.  Returns the rotated Q and K, contiguous;
    with K None, Q alone.

    Q and K may be views whose rows are contiguous (a projection's [B, S, H, D] transposed, a slice of a joint
    projection); ``out`` and ``out_k`` too, and they may be Q and K themselves.  ``positions``: int32, [S] or
    [B, S], None for 0 .. S - 1.  ``inverse`` rotates back, which is the backward pass."""
    args = (Q, K, _frequencies(frequencies), positions, interleaved, magnitude, inverse, out, out_k)
    return calls().rotary(*args) if stream is None else _called(calls().rotary, stream, Q, (out, out_k), args)


def tsa_paged_append(Q, K, V, K_cache, V_cache, page_table, seq_lens, counts=None, frequencies=None, *,
                     interleaved: bool = False, magnitude: float = 1.0, out=None, stream=None):
    """New tokens K, V [B, HK, T, D] to the paged cache K_cache, V_cache [pages, HK, page_size, D]: sequence b
    holds ``seq_lens[b]`` tokens with its ``counts[b]`` (None: T) new ones, the first rows of K and V, which are
    its last tokens.  Token p goes to slot p % page_size of page ``page_table[b, p // page_size]``, K's row
    rotated by its position as by ``tsa_rotary`` (``frequencies`` None: as it is).

    Q [B, H, T, D] is rotated in the same launch, and returned (None for none); its rows that are no tokens --
    past counts, or in front of a sequence shorter than its rows -- become 0.  Q, K, V and ``out`` may be views
    as for ``tsa_rotary``, and ``out`` may be Q."""
    args = (Q, K, V, K_cache, V_cache, page_table, seq_lens, counts, None if frequencies is None else _frequencies(frequencies),
            interleaved, magnitude, out)
    return calls().paged_append(*args) if stream is None else _called(calls().paged_append, stream, K, (out,), args)


def tsa_paged_attention_decode_workspace_bytes(B: int, H: int, HK: int, D: int, page_size: int, max_pages: int,
                                               block: int = 64, nnz_cap: int = 0) -> int:
    return int(lib().tsa_paged_attention_decode_workspace_bytes(B, H, HK, D, page_size, max_pages, block, nnz_cap))


def tsa_paged_attention_decode(Q, K_cache, V_cache, page_table, seq_lens, row_ptr=None, col_idx=None,
                               scale: float | None = None, *, out=None, block: int = 64, workspace=None, stream=None):
    """One new token per sequence: softmax(scale q.k) V of Q [B, H, D] over the ``seq_lens[b]`` tokens that
    sequence b holds in the paged cache (see ``tsa_paged_append``), the new one last; ``scale`` defaults to
    D ** -0.5.  Groups of H / HK heads share a key head.  With ``row_ptr`` and ``col_idx``, row b lists the
    ``block``-token blocks of sequence b that its token visits.  Returns [B, H, D]."""
    args = (Q, K_cache, V_cache, page_table, seq_lens, row_ptr, col_idx, scale, block, out, workspace)
    return calls().paged_decode(*args) if stream is None else _called(calls().paged_decode, stream, Q, (out,), args)
