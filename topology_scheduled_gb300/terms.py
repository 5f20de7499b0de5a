"""Binding of the attentions with learned score terms (include/tsa_terms.h): argument marshalling only.

``tsa_biased_attention*``       -- a learned bias per head and bucket of the distance q - k;
``tsa_differential_attention*`` -- the difference of two softmax maps, weighted by a learned lambda.

Like the calls of ``binding`` they run in libtsa.so on the current stream (or ``stream``) and
raise when a call fails; there is no fallback.
"""
from __future__ import annotations

import math
from array import array

import torch

from .binding import TsaError, _check, _check_qkv, _dtype_code, _lanes_S_D, _made, _on, lib

MAX_BUCKETS = 256


def relative_bucket_starts(num_buckets: int, max_distance: int) -> list[int]:
    """Starts of ``num_buckets`` (even) buckets of the distance q - k: one per distance below
    num_buckets / 2, then borders in geometric steps up to ``max_distance``, the last bucket open.
    Start h + i is the smallest d with d / h >= (max_distance / h) ** (i / h), h = num_buckets / 2,
    found in integer arithmetic."""
    h = num_buckets // 2
    if num_buckets < 2 or num_buckets % 2 or num_buckets > MAX_BUCKETS or max_distance <= h:
        raise ValueError(f"num_buckets must be even, 2 to {MAX_BUCKETS}, and max_distance above half of it")
    starts = list(range(h))
    d = h
    for i in range(h):
        border = max_distance ** i * h ** (h - i)  # d ** h reaches it
        lo, hi = d, max_distance
        while lo < hi:
            mid = (lo + hi) // 2
            lo, hi = (lo, mid) if mid ** h >= border else (mid + 1, hi)
        d = lo
        starts.append(d)
    return starts


def _starts(bucket_starts, bias):
    """The starts as a host array of int32 (the library checks their order)."""
    if isinstance(bucket_starts, torch.Tensor):
        if bucket_starts.is_cuda:
            raise ValueError("bucket_starts must be host integers")
        bucket_starts = bucket_starts.tolist()
    starts = array("i", bucket_starts)
    if bias.shape[-1] != len(starts):
        raise ValueError(f"bias has {bias.shape[-1]} buckets, bucket_starts {len(starts)}")
    return starts, len(starts)


def _schedule(row_ptr, col_idx, rows, device, other):
    """Checks a CSR of `rows` rows; col_idx with at least one entry."""
    for t in (row_ptr, col_idx):
        if t.dtype is not torch.int32 or t.device != device or not t.is_contiguous():
            raise ValueError("row_ptr and col_idx must be contiguous int32 tensors on the inputs' device")
    if row_ptr.numel() != rows + 1:
        raise ValueError(f"row_ptr must hold {rows + 1} entries")
    return col_idx if col_idx.numel() > 0 else _made(other, torch.zeros, 1, dtype=torch.int32, device=device)


def _learned(name, t, shape, like):
    if t.shape != shape or t.dtype is not like.dtype or t.device != like.device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {like.dtype} tensor of shape {tuple(shape)} on {like.device}")


def _output(name, t, like, other):
    """`t`, or a new tensor shaped as `like`."""
    return _made(other, torch.empty_like, like) if t is None else _given(name, t, like.shape, like.dtype, like.device)


def _rows_f32(name, t, shape, device, other):
    return _made(other, torch.empty, shape, dtype=torch.float32, device=device) if t is None else \
        _given(name, t, shape, torch.float32, device)


def _given(name, t, shape, dtype, device):
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t


def _blocks(S, block):
    return -(-S // block) if block > 0 else 0


def _lambda_heads(lambdas, H, D, like):
    """1 (one lambda for all heads) or H; each vector [D / 2], [1, D / 2] or [H, D / 2]."""
    heads = 1 if lambdas[0].dim() == 1 else lambdas[0].shape[0]
    if heads not in (1, H):
        raise ValueError(f"the lambda vectors must be of one head or of {H}")
    for name, t in zip(("lambda_q1", "lambda_k1", "lambda_q2", "lambda_k2"), lambdas):
        _learned(name, t, (D // 2,) if lambdas[0].dim() == 1 else (heads, D // 2), like)
    return heads


def tsa_biased_attention(Q, K, V, row_ptr, col_idx, bias, bucket_starts, scale: float | None = None, *,
                         out=None, block: int = 64, stream=None):
    """Scheduled attention with a learned relative position bias: softmax(scale q.k +
    bias[head, bucket(q - k)]) V over the CSR, in the inputs' type and shape.

    ``bias`` is [H, buckets] of the inputs' type, ``bucket_starts`` the buckets' ascending first
    distances (host integers, the first one 0; see ``relative_bucket_starts``)."""
    return tsa_biased_attention_fwd(Q, K, V, row_ptr, col_idx, bias, bucket_starts, scale, out=out, block=block,
                                    stream=stream, with_lse=False)


def tsa_biased_attention_fwd(Q, K, V, row_ptr, col_idx, bias, bucket_starts, scale: float | None = None, *,
                             out=None, lse=None, block: int = 64, stream=None, with_lse: bool = True):
    """tsa_biased_attention that also returns the rows' log-sum-exp ([B*H, S] float32) for the backward."""
    _check_qkv(Q=Q, K=K, V=V)
    B, H, S, D = _lanes_S_D(Q)
    dev = Q.device
    handle, other = _on(stream, dev)
    ci = _schedule(row_ptr, col_idx, _blocks(S, block), dev, other)
    starts, n = _starts(bucket_starts, bias)
    _learned("bias", bias, (H, n), Q)
    out = _output("out", out, Q, other)
    lse = _rows_f32("lse", lse, (B * H, S), dev, other) if with_lse else None
    _check(lib().tsa_biased_attention_fwd(
        Q.data_ptr(), K.data_ptr(), V.data_ptr(), row_ptr.data_ptr(), ci.data_ptr(), ci.numel(), bias.data_ptr(),
        starts.buffer_info()[0], n, out.data_ptr(), lse.data_ptr() if with_lse else None, _dtype_code(Q), B, H, S, D, block,
        1.0 / math.sqrt(D) if scale is None else float(scale), handle), "tsa_biased_attention_fwd")
    return (out, lse) if with_lse else out


def tsa_differential_attention(Q, K, V, row_ptr, col_idx, lambda_q1, lambda_k1, lambda_q2, lambda_k2,
                               lambda_init: float, scale: float | None = None, *, out=None, block: int = 64,
                               stream=None):
    """Differential attention over the CSR: (softmax(scale q1.k1) - lambda softmax(scale q2.k2)) V,
    in the inputs' type and shape, where q1 | q2 and k1 | k2 are the halves of Q's and K's rows and
    lambda = exp(lambda_q1.lambda_k1) - exp(lambda_q2.lambda_k2) + lambda_init.

    The lambda vectors are [H, D/2] (a lambda per head), [1, D/2] or [D/2] (one for all heads), of
    the inputs' type; ``scale`` defaults to (D/2) ** -0.5."""
    return tsa_differential_attention_fwd(Q, K, V, row_ptr, col_idx, lambda_q1, lambda_k1, lambda_q2, lambda_k2,
                                          lambda_init, scale, out=out, block=block, stream=stream,
                                          for_backward=False)


def tsa_differential_attention_fwd(Q, K, V, row_ptr, col_idx, lambda_q1, lambda_k1, lambda_q2, lambda_k2,
                                   lambda_init: float, scale: float | None = None, *, out=None, out2=None, lse=None,
                                   block: int = 64, stream=None, for_backward: bool = True):
    """tsa_differential_attention that also returns what its backward pass reads: the second map's
    output (shaped as the output) and both maps' log-sum-exp ([2, B*H, S] float32)."""
    _check_qkv(Q=Q, K=K, V=V)
    B, H, S, D = _lanes_S_D(Q)
    dev = Q.device
    handle, other = _on(stream, dev)
    ci = _schedule(row_ptr, col_idx, _blocks(S, block), dev, other)
    lambdas = (lambda_q1, lambda_k1, lambda_q2, lambda_k2)
    heads = _lambda_heads(lambdas, H, D, Q)
    out = _output("out", out, Q, other)
    if for_backward:
        out2 = _output("out2", out2, Q, other)
        lse = _rows_f32("lse", lse, (2, B * H, S), dev, other)
    else:
        out2 = lse = None
    _check(lib().tsa_differential_attention_fwd(
        Q.data_ptr(), K.data_ptr(), V.data_ptr(), row_ptr.data_ptr(), ci.data_ptr(), ci.numel(),
        *(t.data_ptr() for t in lambdas), heads, float(lambda_init), out.data_ptr(),
        out2.data_ptr() if for_backward else None, lse.data_ptr() if for_backward else None, _dtype_code(Q), B, H, S,
        D, block, (D / 2) ** -0.5 if scale is None else float(scale), handle),
        "tsa_differential_attention_fwd")
    return (out, out2, lse) if for_backward else out


def _workspace(t, need, device, where, other):
    if need == 0:
        raise TsaError(2, where)
    if t is None:
        return _made(other, torch.empty, need, dtype=torch.uint8, device=device)
    if t.dtype != torch.uint8 or t.device != device or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on the inputs' device")
    return t


def tsa_biased_attention_backward(Q, K, V, O, dO, lse, row_ptr, col_idx, bias, bucket_starts,
                                  scale: float | None = None, *, block: int = 64, dq=None, dk=None, dv=None,
                                  dbias=None, workspace=None, stream=None):
    """dQ, dK, dV, dbias of tsa_biased_attention for the upstream gradient dO, in the inputs' type;
    O and lse as tsa_biased_attention_fwd returned them."""
    _check_qkv(Q=Q, K=K, V=V, O=O, dO=dO)
    B, H, S, D = _lanes_S_D(Q)
    dev = Q.device
    handle, other = _on(stream, dev)
    ci = _schedule(row_ptr, col_idx, _blocks(S, block), dev, other)
    starts, n = _starts(bucket_starts, bias)
    _learned("bias", bias, (H, n), Q)
    _given("lse", lse, (B * H, S), torch.float32, dev)
    L = lib()
    workspace = _workspace(workspace, int(L.tsa_biased_attention_backward_workspace_bytes(B * H, S, block, ci.numel(), n)),
                           dev, "tsa_biased_attention_backward_workspace_bytes", other)
    dq, dk, dv = (_output(name, t, Q, other) for name, t in (("dq", dq), ("dk", dk), ("dv", dv)))
    dbias = _output("dbias", dbias, bias, other)
    _check(L.tsa_biased_attention_backward(
        Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), dO.data_ptr(), lse.data_ptr(), row_ptr.data_ptr(),
        ci.data_ptr(), ci.numel(), bias.data_ptr(), starts.buffer_info()[0], n, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
        dbias.data_ptr(), _dtype_code(Q), B, H, S, D, block, 1.0 / math.sqrt(D) if scale is None else float(scale),
        workspace.data_ptr(), workspace.numel(), handle),
        "tsa_biased_attention_backward")
    return dq, dk, dv, dbias


def tsa_differential_attention_backward(Q, K, V, O, O2, dO, lse, row_ptr, col_idx, lambda_q1, lambda_k1, lambda_q2,
                                        lambda_k2, lambda_init: float, scale: float | None = None, *,
                                        block: int = 64, dq=None, dk=None, dv=None, dlambdas=None, workspace=None,
                                        stream=None):
    """dQ, dK, dV and the gradients of the four lambda vectors of tsa_differential_attention for the
    upstream gradient dO, in the inputs' type; O, O2 and lse as tsa_differential_attention_fwd
    returned them."""
    _check_qkv(Q=Q, K=K, V=V, O=O, O2=O2, dO=dO)
    B, H, S, D = _lanes_S_D(Q)
    dev = Q.device
    handle, other = _on(stream, dev)
    ci = _schedule(row_ptr, col_idx, _blocks(S, block), dev, other)
    lambdas = (lambda_q1, lambda_k1, lambda_q2, lambda_k2)
    heads = _lambda_heads(lambdas, H, D, Q)
    _given("lse", lse, (2, B * H, S), torch.float32, dev)
    L = lib()
    workspace = _workspace(workspace,
                           int(L.tsa_differential_attention_backward_workspace_bytes(B * H, S, block, ci.numel())), dev,
                           "tsa_differential_attention_backward_workspace_bytes", other)
    dq, dk, dv = (_output(name, t, Q, other) for name, t in (("dq", dq), ("dk", dk), ("dv", dv)))
    dlambdas = [_output("dlambdas", None if dlambdas is None else dlambdas[i], t, other) for i, t in enumerate(lambdas)]
    _check(L.tsa_differential_attention_backward(
        Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), O2.data_ptr(), dO.data_ptr(), lse.data_ptr(),
        row_ptr.data_ptr(), ci.data_ptr(), ci.numel(), *(t.data_ptr() for t in lambdas), heads, float(lambda_init),
        dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), *(t.data_ptr() for t in dlambdas), _dtype_code(Q), B, H, S, D,
        block, (D / 2) ** -0.5 if scale is None else float(scale), workspace.data_ptr(), workspace.numel(),
        handle), "tsa_differential_attention_backward")
    return (dq, dk, dv, *dlambdas)


def _cache(Q, K, V, seq_lens):
    """B, H, capacity, D of a decode call's tensors."""
    if Q.dim() != 3 or not Q.is_cuda or not Q.is_contiguous():
        raise ValueError("Q must be a contiguous CUDA tensor [B, H, D]")
    B, H, D = Q.shape
    for name, t in (("K", K), ("V", V)):
        if t.dim() != 4 or t.shape != (B, H, K.shape[2], D) or t.dtype != Q.dtype or t.device != Q.device or \
                not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [B, H, capacity, D] tensor of Q's type and device")
    if seq_lens.dtype != torch.int32 or seq_lens.shape != (B,) or seq_lens.device != Q.device or \
            not seq_lens.is_contiguous():
        raise ValueError("seq_lens must be a contiguous int32 tensor [B] on the inputs' device")
    return B, H, K.shape[2], D


def tsa_biased_attention_decode(Q, K, V, seq_lens, row_ptr, col_idx, bias, bucket_starts, scale: float | None = None,
                                *, out=None, block: int = 64, stream=None):
    """One new token per sequence: Q [B, H, D] against the cache K, V [B, H, capacity, D], whose first
    ``seq_lens[b]`` tokens are sequence b's, the new one last.  Row b of the CSR lists the cache blocks
    that sequence b's token visits; scores as in tsa_biased_attention.  Returns [B, H, D]."""
    B, H, cap, D = _cache(Q, K, V, seq_lens)
    handle, other = _on(stream, Q.device)
    ci = _schedule(row_ptr, col_idx, B, Q.device, other)
    starts, n = _starts(bucket_starts, bias)
    _learned("bias", bias, (H, n), Q)
    out = _output("out", out, Q, other)
    _check(lib().tsa_biased_attention_decode(
        Q.data_ptr(), K.data_ptr(), V.data_ptr(), seq_lens.data_ptr(), row_ptr.data_ptr(), ci.data_ptr(), ci.numel(),
        bias.data_ptr(), starts.buffer_info()[0], n, out.data_ptr(), _dtype_code(Q), B, H, cap, D, block,
        1.0 / math.sqrt(D) if scale is None else float(scale), handle), "tsa_biased_attention_decode")
    return out


def tsa_differential_attention_decode(Q, K, V, seq_lens, row_ptr, col_idx, lambda_q1, lambda_k1, lambda_q2, lambda_k2,
                                      lambda_init: float, scale: float | None = None, *, out=None, block: int = 64,
                                      stream=None):
    """One new token per sequence, as tsa_biased_attention_decode, with the two maps of
    tsa_differential_attention."""
    B, H, cap, D = _cache(Q, K, V, seq_lens)
    handle, other = _on(stream, Q.device)
    ci = _schedule(row_ptr, col_idx, B, Q.device, other)
    lambdas = (lambda_q1, lambda_k1, lambda_q2, lambda_k2)
    heads = _lambda_heads(lambdas, H, D, Q)
    out = _output("out", out, Q, other)
    _check(lib().tsa_differential_attention_decode(
        Q.data_ptr(), K.data_ptr(), V.data_ptr(), seq_lens.data_ptr(), row_ptr.data_ptr(), ci.data_ptr(), ci.numel(),
        *(t.data_ptr() for t in lambdas), heads, float(lambda_init), out.data_ptr(), _dtype_code(Q), B, H, cap, D,
        block, (D / 2) ** -0.5 if scale is None else float(scale), handle),
        "tsa_differential_attention_decode")
    return out
