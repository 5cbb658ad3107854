"""The training-step operators as differentiable functions of torch tensors.

Each pairs an operator of :mod:`all_gather_gb300.ops` with its gradient; the
forward pass keeps what the gradient reads and nothing else: the inputs of the
head norm (its statistics are computed again), the hidden states, weight and
log-sums of the cross entropy (the logits are computed again), and the 8-bit
codes of a SwiGLU's gate and up (the inputs themselves are not kept).
"""
from __future__ import annotations

import torch

from . import ops


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, table, positions, q_weight, k_weight, eps, interleaved):
        ctx.save_for_backward(q, k, table, positions, q_weight, k_weight)
        ctx.how = eps, interleaved
        return ops.qk_norm_rope(q, k, table, positions, q_weight, k_weight, eps, interleaved)

    @staticmethod
    def backward(ctx, dq, dk):
        q, k, table, positions, q_weight, k_weight = ctx.saved_tensors
        dq, dk, dqw, dkw = ops.qk_norm_rope_grad(_rows(dq), _rows(dk), q, k, table, positions, q_weight, k_weight,
                                                 *ctx.how)
        return dq, dk, None, None, dqw, dkw, None, None


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, targets, ignore_index):
        loss, lse = ops.linear_cross_entropy(x, weight, targets, ignore_index)
        ctx.save_for_backward(x, weight, targets, lse)
        ctx.ignore_index = ignore_index
        return loss

    @staticmethod
    def backward(ctx, dloss):
        x, weight, targets, lse = ctx.saved_tensors
        dx, dw = ops.linear_cross_entropy_grad(x, weight, targets, lse, dloss.contiguous(), ctx.ignore_index)
        return dx, dw, None, None


class _SwigluCkpt8(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate, up):
        h, ckpt = ops.swiglu_ckpt8(gate, up)
        ctx.save_for_backward(*ckpt)
        return h

    @staticmethod
    def backward(ctx, dh):
        dgate, dup, _ = ops.swiglu_ckpt8_grad(ops.Ckpt8(*ctx.saved_tensors), _rows(dh), need_h=False)
        return dgate, dup


def _rows(t):
    """An incoming gradient with contiguous rows (autograd hands out expanded ones)."""
    return t if t.stride(-1) == 1 or t.shape[-1] <= 1 else t.contiguous()


def qk_norm_rope(q, k, table=None, positions=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False):
    """:func:`ops.qk_norm_rope`, differentiable in q, k and the weights."""
    return _QkNormRope.apply(q, k, table, positions, q_weight, k_weight, eps, interleaved)


def linear_cross_entropy(x, weight, targets, ignore_index: int = -100):
    """The losses [T] of :func:`ops.linear_cross_entropy`, differentiable in x and weight."""
    return _LinearCrossEntropy.apply(x, weight, targets, ignore_index)


def swiglu(gate, up):
    """silu(gate) * up, differentiable, keeping gate and up in 8 bits for the backward pass (so its gradients are those
    at the 8-bit values)."""
    return _SwigluCkpt8.apply(gate, up)
