"""torch.autograd wrappers over the scheduled-attention kernels (argument plumbing only).

``scheduled_attention(Q, K, V, row_ptr, col_idx, scale, block=64)`` runs
tsa_scheduled_attention_fwd and keeps its log-sum-exp; its backward runs
tsa_scheduled_attention_backward (blocks of 64 or 128 tokens).  The CSR is not differentiable.

``biased_attention`` and ``differential_attention`` do the same for the attentions with learned
score terms; their learned inputs get gradients as well.  ``rotary`` rotates Q and K by their
positions, and their gradients back.

Capturing a backward pass into a CUDA graph: PyTorch's accumulation nodes keep the stream they were
made on, so the captured pass needs leaves of its own (or torch.autograd.grad, which accumulates
nothing) while an eager graph of the same leaves is alive.
"""
from __future__ import annotations

import torch

from .binding import calls, tsa_scheduled_attention_backward, tsa_scheduled_attention_fwd
from .cache import _frequencies
from .terms import (_starts, tsa_biased_attention_backward, tsa_biased_attention_fwd,
                    tsa_differential_attention_backward, tsa_differential_attention_fwd)


def _dense(t):
    """`t` as the kernels read it: contiguous, from a 16-byte boundary on.  (The gradient that reaches a
    backward pass may be a slice of another, at any element.)"""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class ScheduledAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, Q, K, V, row_ptr, col_idx, scale, block):
        Q, K, V = (_dense(t) for t in (Q, K, V))
        O, lse = tsa_scheduled_attention_fwd(Q, K, V, row_ptr, col_idx, scale, block=block)
        ctx.save_for_backward(Q, K, V, O, lse, row_ptr, col_idx)
        ctx.scale = scale
        ctx.block = block
        return O

    @staticmethod
    def backward(ctx, dO):
        Q, K, V, O, lse, row_ptr, col_idx = ctx.saved_tensors
        dQ, dK, dV = tsa_scheduled_attention_backward(Q, K, V, O, _dense(dO), lse, row_ptr, col_idx,
                                                      ctx.scale, block=ctx.block)
        return dQ, dK, dV, None, None, None, None


def scheduled_attention(Q, K, V, row_ptr, col_idx, scale: float | None = None, block: int = 64):
    if scale is None:
        scale = Q.shape[-1] ** -0.5
    return ScheduledAttention.apply(Q, K, V, row_ptr, col_idx, float(scale), int(block))


class BiasedAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, Q, K, V, row_ptr, col_idx, bias, bucket_starts, scale, block):
        Q, K, V, bias = _dense(Q), _dense(K), _dense(V), bias.contiguous()
        bucket_starts, _ = _starts(bucket_starts, bias)  # a copy: the caller's may change before the backward
        O, lse = tsa_biased_attention_fwd(Q, K, V, row_ptr, col_idx, bias, bucket_starts, scale, block=block)
        ctx.save_for_backward(Q, K, V, O, lse, row_ptr, col_idx, bias)
        ctx.settings = bucket_starts, scale, block
        return O

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dO):
        Q, K, V, O, lse, row_ptr, col_idx, bias = ctx.saved_tensors
        bucket_starts, scale, block = ctx.settings
        dQ, dK, dV, dbias = tsa_biased_attention_backward(Q, K, V, O, _dense(dO), lse, row_ptr, col_idx, bias,
                                                          bucket_starts, scale, block=block)
        return dQ, dK, dV, None, None, dbias, None, None, None


def biased_attention(Q, K, V, row_ptr, col_idx, bias, bucket_starts, scale: float | None = None, block: int = 64):
    """tsa_biased_attention with gradients for Q, K, V and bias (blocks of 64 or 128 tokens)."""
    return BiasedAttention.apply(Q, K, V, row_ptr, col_idx, bias, bucket_starts, scale, int(block))


class DifferentialAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, Q, K, V, row_ptr, col_idx, lambda_q1, lambda_k1, lambda_q2, lambda_k2, lambda_init, scale, block):
        Q, K, V = (_dense(t) for t in (Q, K, V))
        lambdas = [t.contiguous() for t in (lambda_q1, lambda_k1, lambda_q2, lambda_k2)]
        O, O2, lse = tsa_differential_attention_fwd(Q, K, V, row_ptr, col_idx, *lambdas, lambda_init, scale, block=block)
        ctx.save_for_backward(Q, K, V, O, O2, lse, row_ptr, col_idx, *lambdas)
        ctx.settings = lambda_init, scale, block
        return O

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dO):
        Q, K, V, O, O2, lse, row_ptr, col_idx, *lambdas = ctx.saved_tensors
        lambda_init, scale, block = ctx.settings
        grads = tsa_differential_attention_backward(Q, K, V, O, O2, _dense(dO), lse, row_ptr, col_idx, *lambdas,
                                                    lambda_init, scale, block=block)
        return (*grads[:3], None, None, *grads[3:], None, None, None)


def differential_attention(Q, K, V, row_ptr, col_idx, lambda_q1, lambda_k1, lambda_q2, lambda_k2, lambda_init: float,
                           scale: float | None = None, block: int = 64):
    """tsa_differential_attention with gradients for Q, K, V and the four lambda vectors (blocks of
    64 or 128 tokens)."""
    return DifferentialAttention.apply(Q, K, V, row_ptr, col_idx, lambda_q1, lambda_k1, lambda_q2, lambda_k2,
                                       float(lambda_init), scale, int(block))


def rotary(Q, K, frequencies, positions=None, interleaved: bool = False, magnitude: float = 1.0):
    """tsa_rotary of Q and K (or of Q alone, K None) with gradients for both, in their layouts."""
    return calls().rotary_autograd(Q, K, _frequencies(frequencies), positions, interleaved, magnitude)
