"""The training-step operators as differentiable functions of torch tensors.

Each pairs an operator of :mod:`all_gather_gb300.ops` with its gradient; the
forward pass keeps what the gradient reads and nothing else: the inputs of the
head norm (its statistics are computed again), the hidden states, weight and
log-sums of the cross entropy (the logits are computed again), the 8-bit codes
of a SwiGLU's gate and up (the inputs themselves are not kept), the heads,
output and log-sums of the attention (the scores are computed again), and the
rows and parameters of the layer norm (its statistics are computed again).

They can be differentiated once: a gradient taken with ``create_graph`` raises
an error when it is differentiated itself.
"""
from __future__ import annotations

import torch

from . import ops


class _Once(torch.autograd.Function):
    """Gradients of a backward pass that is recorded itself: they depend on `links`, and going through them again is an
    error.  (once_differentiable lets it pass where the incoming gradients are constants.)"""

    @staticmethod
    def forward(ctx, n, *grads_and_links):
        return grads_and_links[:n]

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("all_gather_gb300.autograd: the operators have no second derivatives")


def _once(grads, *links):
    """What a backward pass returns, None among it; links: tensors that the gradients depend on."""
    if not torch.is_grad_enabled():  # not recorded
        return grads
    some = [g for g in grads if g is not None]
    passed = iter(_Once.apply(len(some), *some, *[t for t in links if t is not None]))
    return tuple(None if g is None else next(passed) for g in grads)


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, table, positions, q_weight, k_weight, eps, interleaved):
        if ctx.needs_input_grad[2]:
            raise ValueError("table has no gradient here, and requires one")
        ctx.save_for_backward(q, k, table, positions, q_weight, k_weight)
        ctx.how = eps, interleaved
        return ops.qk_norm_rope(q, k, table, positions, q_weight, k_weight, eps, interleaved)

    @staticmethod
    def backward(ctx, dq, dk):
        given = dq, dk
        q, k, table, positions, q_weight, k_weight = ctx.saved_tensors
        dq, dk, dqw, dkw = ops.qk_norm_rope_grad(_rows(dq), _rows(dk), q, k, table, positions, q_weight, k_weight,
                                                 *ctx.how)
        return _once((dq, dk, None, None, dqw, dkw, None, None), *given, q, k, q_weight, k_weight)


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, targets, ignore_index, workspace):
        loss, lse = ops.linear_cross_entropy(x, weight, targets, ignore_index, workspace=workspace)
        ctx.save_for_backward(x, weight, targets, lse)
        ctx.ignore_index = ignore_index
        ctx.set_materialize_grads(False)
        return loss, lse

    @staticmethod
    def backward(ctx, dloss, dlse):
        if dlse is not None:
            raise RuntimeError("all_gather_gb300.autograd: lse has no gradient, the loss has")
        if dloss is None:
            return None, None, None, None, None
        x, weight, targets, lse = ctx.saved_tensors
        dx, dw = ops.linear_cross_entropy_grad(x, weight, targets, lse, dloss.contiguous(), ctx.ignore_index)
        return _once((dx, dw, None, None, None), dloss, x, weight)


class _SwigluCkpt8(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate, up):
        h, ckpt = ops.swiglu_ckpt8(gate, up)
        link = h.new_empty(0)  # an output, so that it leads to gate and up, which are not kept
        ctx.save_for_backward(*ckpt, link)
        ctx.mark_non_differentiable(*ckpt)
        return h, link, *ckpt

    @staticmethod
    def backward(ctx, dh, *_):
        *ckpt, link = ctx.saved_tensors
        dgate, dup, _ = ops.swiglu_ckpt8_grad(ops.Ckpt8(*ckpt), _rows(dh), need_h=False)
        return _once((dgate, dup), dh, link)


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, offsets, causal, scale):
        o, lse = ops.attention(q, k, v, offsets, causal, scale)
        ctx.save_for_backward(q, k, v, offsets, o, lse)
        ctx.how = causal, scale
        ctx.set_materialize_grads(False)
        return o, lse

    @staticmethod
    def backward(ctx, do, dlse):
        if dlse is not None:
            raise RuntimeError("all_gather_gb300.autograd: lse has no gradient, the attention's output has")
        if do is None:
            return None, None, None, None, None, None
        q, k, v, offsets, o, lse = ctx.saved_tensors
        grads = ops.attention_grad(_head_rows(do), q, k, v, o, lse, offsets, *ctx.how)
        return _once((*grads, None, None, None), do, q, k, v)


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, center):
        ctx.save_for_backward(x, weight, bias)
        ctx.how = eps, center
        return ops.layer_norm(x, weight, bias, eps, center)

    @staticmethod
    def backward(ctx, dy):
        x, weight, bias = ctx.saved_tensors
        grads = ops.layer_norm_grad(_rows(dy), x, weight, bias, *ctx.how)
        return _once((*grads, None, None), dy, x, weight, bias)


def _head_rows(t):
    """An incoming gradient of heads with rows on 16-byte boundaries."""
    st = t.stride()
    if st[2] == 1 and st[0] > 0 and st[1] > 0 and not (st[0] % 8 or st[1] % 8 or t.data_ptr() % 16):
        return t
    return t.clone(memory_format=torch.contiguous_format)


def _rows(t):
    """An incoming gradient with contiguous rows (autograd hands out expanded ones)."""
    return t if t.stride(-1) == 1 or t.shape[-1] <= 1 else t.contiguous()


def qk_norm_rope(q, k, table=None, positions=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False):
    """:func:`ops.qk_norm_rope`, differentiable in q, k and the weights."""
    return _QkNormRope.apply(q, k, table, positions, q_weight, k_weight, eps, interleaved)


def linear_cross_entropy(x, weight, targets, ignore_index: int = -100):
    """The losses [T] of :func:`ops.linear_cross_entropy`, differentiable in x and weight."""
    return loss_and_lse(x, weight, targets, ignore_index)[0]


def loss_and_lse(x, weight, targets, ignore_index: int = -100, workspace=None):
    """(loss, lse) of :func:`ops.linear_cross_entropy`, the loss differentiable in x and weight; a gradient of lse is
    refused."""
    return _LinearCrossEntropy.apply(x, weight, targets, ignore_index, workspace)


def swiglu_and_ckpt8(gate, up):
    """(h, ckpt) of :func:`ops.swiglu_ckpt8`, h differentiable in gate and up as :func:`swiglu` is; the codes are not."""
    h, _, *ckpt = _SwigluCkpt8.apply(gate, up)
    return h, ops.Ckpt8(*ckpt)


def swiglu(gate, up):
    """silu(gate) * up, differentiable, keeping gate and up in 8 bits for the backward pass (so its gradients are those
    at the 8-bit values)."""
    return _SwigluCkpt8.apply(gate, up)[0]


def attention(q, k, v, offsets=None, causal: bool = True, scale=None):
    """The output of :func:`ops.attention`, differentiable in q, k and v."""
    return attention_and_lse(q, k, v, offsets, causal, scale)[0]


def attention_and_lse(q, k, v, offsets=None, causal: bool = True, scale=None):
    """(o, lse) of :func:`ops.attention`, o differentiable in q, k and v; a gradient of lse is refused."""
    return _Attention.apply(q, k, v, offsets, causal, scale)


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, center: bool = True):
    """:func:`ops.layer_norm`, differentiable in x, weight and bias."""
    return _LayerNorm.apply(x, weight, bias, eps, center)
