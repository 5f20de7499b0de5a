"""Binding of the rotary positions, the paged key/value cache and its one-token attention
(include/tsa_cache.h): argument marshalling only.

``tsa_rotary``                 -- rotates the pairs of Q's and K's rows by their positions (or back);
``tsa_paged_append``           -- writes new tokens to a paged cache, rotating on the way;
``tsa_paged_attention_decode`` -- one new token per sequence against a paged cache.

Like the calls of ``binding`` they run in libtsa.so on the current stream (or ``stream``) and
raise when a call fails; there is no fallback.
"""
from __future__ import annotations

import math
from array import array
from functools import lru_cache

import torch

from .binding import _check, _dtype_code, _made, _on, lib
from .terms import _given, _output, _schedule, _workspace

_NONE = (0, 0, 0)


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                       original_length: int | None = None, low: float = 1.0, high: float = 32.0) -> array:
    """The angle per position of each of the rotary_dim / 2 pairs, base ** (-2 i / rotary_dim), in 64 bits.

    ``scaling`` for contexts ``factor`` times as long as the ``original_length`` tokens trained on:
    ``"linear"`` divides every frequency by factor; ``"base"`` enlarges the base to
    base * factor ** (rotary_dim / (rotary_dim - 2)), which divides the last pair's by factor and leaves the
    first pair's; ``"ramp"`` divides the pairs that turn less than ``low`` times in original_length tokens,
    leaves those that turn more than ``high`` times, and blends linearly between (its attention is sharpened
    by ``rotary_magnitude``)."""
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


def _rows(name, t, like=None):
    """Checks a tensor [B, heads, tokens, D] whose rows are contiguous, on `like`'s device and of its type, batch,
    tokens and D."""
    shape = t.shape
    if len(shape) != 4 or not t.is_cuda or t.stride(3) != 1:
        raise ValueError(f"{name} must be a CUDA tensor [B, heads, tokens, D] with contiguous rows")
    if like is not None:
        other = like.shape
        if t.dtype is not like.dtype or t.device != like.device or shape[0] != other[0] or shape[2] != other[2] or \
                shape[3] != other[3]:
            raise ValueError(f"{name} must have the type, device, batch, tokens and row length of the others")


def _rotated(name, t, like, other):
    """`t`, or a new contiguous tensor shaped as `like`."""
    if t is None:
        return _made(other, torch.empty_like, like, memory_format=torch.contiguous_format)
    _rows(name, t, like)
    if t.shape != like.shape:
        raise ValueError(f"{name} must have the shape {tuple(like.shape)}")
    return t


def tsa_rotary(Q, K, frequencies, positions=None, *, interleaved: bool = False, magnitude: float = 1.0,
               inverse: bool = False, out=None, out_k=None, stream=None):
    """Rotary positions: every pair of the first 2 len(frequencies) dimensions of the rows of Q [B, H, S, D] and
    K [B, HK, S, D] is rotated by position * frequency and scaled by ``magnitude``; the rest is copied.  The
    pairs are (i, i + R/2), or (2 i, 2 i + 1) if ``interleaved``.  Returns the rotated Q and K, contiguous;
    with K None, Q alone.

    Q and K may be views whose rows are contiguous (a projection's [B, S, H, D] transposed, a slice of a joint
    projection); ``out`` and ``out_k`` too, and they may be Q and K themselves.  ``positions``: int32, [S] or
    [B, S], None for 0 .. S - 1.  ``inverse`` rotates back, which is the backward pass."""
    _rows("Q", Q)
    B, H, S, D = Q.shape
    dev = Q.device
    handle, other = _on(stream, dev)
    if K is not None:
        _rows("K", K, Q)
    elif out_k is not None:
        raise ValueError("out_k without K")
    f = _frequencies(frequencies)
    if positions is not None:
        if positions.dtype is not torch.int32 or positions.device != dev or not positions.is_contiguous() or \
                positions.shape not in ((S,), (B, S)):
            raise ValueError("positions must be a contiguous int32 tensor [S] or [B, S] on the inputs' device")
    out = _rotated("out", out, Q, other)
    if K is not None:
        out_k = _rotated("out_k", out_k, K, other)
    at, rows = (None, 1) if positions is None else (positions.data_ptr(), 1 if positions.dim() == 1 else B)
    if K is None:
        strides = array("q", Q.stride()[:3] + _NONE + out.stride()[:3] + _NONE)
        _check(lib().tsa_rotary(
            Q.data_ptr(), None, strides.buffer_info()[0], at, rows, f.buffer_info()[0], 2 * len(f), interleaved, magnitude,
            inverse, out.data_ptr(), None, _dtype_code(Q), B, H, 0, S, D, handle), "tsa_rotary")
        return out
    strides = array("q", Q.stride()[:3] + K.stride()[:3] + out.stride()[:3] + out_k.stride()[:3])
    _check(lib().tsa_rotary(
        Q.data_ptr(), K.data_ptr(), strides.buffer_info()[0], at, rows, f.buffer_info()[0], 2 * len(f), interleaved,
        magnitude, inverse, out.data_ptr(), out_k.data_ptr(), _dtype_code(Q), B, H, K.shape[1], S, D, handle), "tsa_rotary")
    return out, out_k


def _pages(K_cache, V_cache, page_table, seq_lens, B, HK, D, like):
    """Checks a paged cache [pages, HK, page_size, D] and its lists; page counts, sizes and strides."""
    shape = K_cache.shape
    if len(shape) != 4 or shape[1] != HK or shape[3] != D:
        raise ValueError(f"K_cache must be [pages, {HK}, page_size, {D}]")
    inner = (shape[2] * D, D, 1)
    for name, t in (("K_cache", K_cache), ("V_cache", V_cache)):
        if t.shape != shape or t.dtype is not like.dtype or t.device != like.device or t.stride()[1:] != inner:
            raise ValueError(f"{name} must be a [pages, HK, page_size, D] tensor of the inputs' type and device, "
                             "its pages contiguous")
    if page_table.dim() != 2 or page_table.shape[0] != B or page_table.dtype is not torch.int32 or \
            page_table.device != like.device or not page_table.is_contiguous():
        raise ValueError("page_table must be a contiguous int32 tensor [B, pages] on the inputs' device")
    _given("seq_lens", seq_lens, (B,), torch.int32, like.device)
    return shape[0], shape[2], K_cache.stride(0), V_cache.stride(0)


def tsa_paged_append(Q, K, V, K_cache, V_cache, page_table, seq_lens, counts=None, frequencies=None, *,
                     interleaved: bool = False, magnitude: float = 1.0, out=None, stream=None):
    """New tokens K, V [B, HK, T, D] to the paged cache K_cache, V_cache [pages, HK, page_size, D]: sequence b
    holds ``seq_lens[b]`` tokens with its ``counts[b]`` (None: T) new ones, the first rows of K and V, which are
    its last tokens.  Token p goes to slot p % page_size of page ``page_table[b, p // page_size]``, K's row
    rotated by its position as by ``tsa_rotary`` (``frequencies`` None: as it is).

    Q [B, H, T, D] is rotated in the same launch, and returned (None for none); its rows that are no tokens --
    past counts, or in front of a sequence shorter than its rows -- become 0.  Q, K, V and ``out`` may be views
    as for ``tsa_rotary``, and ``out`` may be Q."""
    _rows("K", K)
    B, HK, T, D = K.shape
    _rows("V", V, K)
    if V.shape != K.shape:
        raise ValueError("V must have K's shape")
    handle, other = _on(stream, K.device)
    if Q is not None:
        _rows("Q", Q, K)
        if frequencies is None:
            raise ValueError("Q is there to be rotated: frequencies are missing")
        out = _rotated("out", out, Q, other)
    elif out is not None:
        raise ValueError("out without Q")
    num, size, k_stride, v_stride = _pages(K_cache, V_cache, page_table, seq_lens, B, HK, D, K)
    if counts is not None:
        _given("counts", counts, (B,), torch.int32, K.device)
    f = None if frequencies is None else _frequencies(frequencies)
    strides = array("q", (_NONE if Q is None else Q.stride()[:3]) + K.stride()[:3] + V.stride()[:3] +
                    (_NONE if Q is None else out.stride()[:3]))
    _check(lib().tsa_paged_append(
        None if Q is None else Q.data_ptr(), K.data_ptr(), V.data_ptr(), strides.buffer_info()[0], K_cache.data_ptr(),
        V_cache.data_ptr(), num, size, k_stride, v_stride, page_table.data_ptr(), page_table.shape[1],
        seq_lens.data_ptr(), None if counts is None else counts.data_ptr(), None if f is None else f.buffer_info()[0],
        0 if f is None else 2 * len(f), interleaved, magnitude, None if Q is None else out.data_ptr(), _dtype_code(K),
        B, 0 if Q is None else Q.shape[1], HK, T, D, handle), "tsa_paged_append")
    return out


@lru_cache(maxsize=1024)  # of sizes alone
def tsa_paged_attention_decode_workspace_bytes(B: int, H: int, HK: int, D: int, page_size: int, max_pages: int,
                                               block: int = 64, nnz_cap: int = 0) -> int:
    return int(lib().tsa_paged_attention_decode_workspace_bytes(B, H, HK, D, page_size, max_pages, block, nnz_cap))


def tsa_paged_attention_decode(Q, K_cache, V_cache, page_table, seq_lens, row_ptr=None, col_idx=None,
                               scale: float | None = None, *, out=None, block: int = 64, workspace=None, stream=None):
    """One new token per sequence: softmax(scale q.k) V of Q [B, H, D] over the ``seq_lens[b]`` tokens that
    sequence b holds in the paged cache (see ``tsa_paged_append``), the new one last; ``scale`` defaults to
    D ** -0.5.  Groups of H / HK heads share a key head.  With ``row_ptr`` and ``col_idx``, row b lists the
    ``block``-token blocks of sequence b that its token visits.  Returns [B, H, D]."""
    if Q.dim() != 3 or not Q.is_cuda or not Q.is_contiguous():
        raise ValueError("Q must be a contiguous CUDA tensor [B, H, D]")
    B, H, D = Q.shape
    HK = K_cache.shape[1] if K_cache.dim() == 4 else 0
    handle, other = _on(stream, Q.device)
    num, size, k_stride, v_stride = _pages(K_cache, V_cache, page_table, seq_lens, B, HK, D, Q)
    if (row_ptr is None) != (col_idx is None):
        raise ValueError("row_ptr and col_idx go together")
    ci = None if row_ptr is None else _schedule(row_ptr, col_idx, B, Q.device, other)
    nnz = 0 if ci is None else ci.numel()
    out = _output("out", out, Q, other)
    need = tsa_paged_attention_decode_workspace_bytes(B, H, HK, D, size, page_table.shape[1], block, nnz)
    if need or workspace is not None:
        workspace = _workspace(workspace, max(need, 1), Q.device, "tsa_paged_attention_decode", other)
    _check(lib().tsa_paged_attention_decode(
        Q.data_ptr(), K_cache.data_ptr(), V_cache.data_ptr(), num, size, k_stride, v_stride, page_table.data_ptr(),
        page_table.shape[1], seq_lens.data_ptr(), None if ci is None else row_ptr.data_ptr(),
        None if ci is None else ci.data_ptr(), nnz, out.data_ptr(), _dtype_code(Q), B, H, HK, D, block,
        1.0 / math.sqrt(D) if scale is None else float(scale), None if workspace is None else workspace.data_ptr(),
        0 if workspace is None else workspace.numel(), handle), "tsa_paged_attention_decode")
    return out
