"""Training-step operators on torch tensors: the compute next to the
collectives of an FSDP2 step.

Thin wrappers of the ``tide_*`` entry points of the same names
(``include/tide.h`` has the formulas): they check types and shapes, allocate
the outputs that are not passed in ``out`` and the scratch memory, and launch
on ``stream`` (default: the current stream).  Nothing is computed in Python.
A tensor that another stream may still be using is the caller's to order, as
with any asynchronous call; tensors allocated here belong to the current
stream, so pass ``out`` and ``workspace`` to run on another one.

Every operator has its gradient as a function of its own that takes and
returns plain tensors; gradients of parameters have the parameter's type and
can be written straight into a gradient arena with ``out``.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import _binding as _b

_DTYPES = {torch.bfloat16: _b.TIDE_DTYPE_BF16, torch.float32: _b.TIDE_DTYPE_F32}
_INT_BYTES = {torch.int32: 4, torch.int64: 8}
ROPE_SCALINGS = {None: 0, "linear": 1, "by_parts": 2}


def _stream(stream) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream if isinstance(stream, int) else stream.cuda_stream


def _dtype(t, name):
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError(f"{name} is {t.dtype}: need bfloat16 or float32")
    return dt


def _on_device(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} is not on a CUDA device")


def _like(t, ref, shape, name):
    """Checks an output or companion tensor: ref's type and device, this shape, contiguous rows."""
    if t.dtype != ref.dtype or t.device != ref.device:
        raise TypeError(f"{name} is {t.dtype} on {t.device}, expected {ref.dtype} on {ref.device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name} has no contiguous last dimension")


def _workspace(n: int, workspace, device):
    """(tensor that keeps it alive, pointer, bytes) of scratch memory."""
    if workspace is None:
        workspace = torch.empty(n, dtype=torch.uint8, device=device)
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


# ------------------------------------------------------------------ head norm with rotation

def rope_table(max_position: int, rotary_dim: int, base: float = 10000.0, scaling: Optional[str] = None,
               factor: float = 1.0, low_freq_factor: float = 1.0, high_freq_factor: float = 4.0,
               original: float = 8192.0, device=None, out=None, stream=None):
    """fp32 [max_position, rotary_dim]: cosines, then sines, of every position's angles.
    ``scaling``: None, "linear" (positions divided by ``factor``) or "by_parts"."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling {scaling!r}: need one of {list(ROPE_SCALINGS)}")
    if out is None:
        out = torch.empty((max_position, rotary_dim), dtype=torch.float32, device=device or "cuda")
    elif (out.dtype != torch.float32 or not out.is_cuda or not out.is_contiguous()
          or tuple(out.shape) != (max_position, rotary_dim)):
        raise ValueError(f"out must be a contiguous float32 CUDA tensor [{max_position}, {rotary_dim}]")
    _b.tide_rope_table(max_position, rotary_dim, base, ROPE_SCALINGS[scaling], factor, low_freq_factor,
                       high_freq_factor, original, out.data_ptr(), _stream(stream))
    return out


def _heads(t, name):
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    if t.stride(2) != 1 and t.shape[2] > 1:
        raise ValueError(f"{name} has no contiguous last dimension")
    return _b.Heads(t.data_ptr(), t.stride(0), t.stride(1))


def _qk_desc(q, k, table, positions, q_weight, k_weight, eps, interleaved):
    dt = _dtype(q, "q")
    _on_device(q, "q")
    T, Hq, D = q.shape
    if k.dtype != q.dtype or k.device != q.device or k.shape[0] != T or k.shape[2] != D:
        raise ValueError("q and k must agree in type, device, tokens and head_dim")
    R = 0
    if table is not None:
        if table.dtype != torch.float32 or table.dim() != 2 or not table.is_contiguous() or table.device != q.device:
            raise ValueError("table must be a contiguous float32 tensor [positions, rotary_dim] on q's device")
        R = table.shape[1]
        if positions is None or positions.dtype not in _INT_BYTES or positions.device != q.device:
            raise ValueError("positions must be an int32 or int64 tensor on q's device")
        if tuple(positions.shape) != (T,) or (T > 1 and positions.stride(0) != 1):
            raise ValueError(f"positions must be contiguous of shape ({T},)")
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _like(w, q, (D,), name)
    return _b.QkDesc(T, Hq, k.shape[1], D, R, table.shape[0] if R else 0, table.data_ptr() if R else None,
                     positions.data_ptr() if R else None, _INT_BYTES[positions.dtype] if R else 8, dt,
                     int(bool(interleaved)), eps, None if q_weight is None else q_weight.data_ptr(),
                     None if k_weight is None else k_weight.data_ptr())


def qk_norm_rope(q, k, table=None, positions=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False, out=None, stream=None):
    """(q_out, k_out): queries [T, Hq, D] and keys [T, Hk, D] normed for each head (where a weight [D] is given) and
    their first ``table.shape[1]`` columns rotated by the angles of ``positions`` [T] (where a table is given).
    ``out = (q_out, k_out)`` may be (q, k) themselves."""
    qh, kh = _heads(q, "q"), _heads(k, "k")
    desc = _qk_desc(q, k, table, positions, q_weight, k_weight, eps, interleaved)
    if out is None:
        q_out, k_out = torch.empty(q.shape, dtype=q.dtype, device=q.device), torch.empty(k.shape, dtype=k.dtype,
                                                                                         device=k.device)
    else:
        q_out, k_out = out
        _like(q_out, q, q.shape, "q_out")
        _like(k_out, k, k.shape, "k_out")
    _b.tide_qk_norm_rope(desc, qh, kh, _heads(q_out, "q_out"), _heads(k_out, "k_out"), _stream(stream))
    return q_out, k_out


def qk_norm_rope_grad(dq_out, dk_out, q, k, table=None, positions=None, q_weight=None, k_weight=None,
                      eps: float = 1e-6, interleaved: bool = False, out=None, workspace=None, stream=None):
    """(dq, dk, dq_weight, dk_weight) of :func:`qk_norm_rope` from its outputs' gradients and its inputs.  A weight
    that is None has no gradient (None), and its ``q`` or ``k`` is used for its shape only."""
    desc = _qk_desc(q, k, table, positions, q_weight, k_weight, eps, interleaved)
    _like(dq_out, q, q.shape, "dq_out")
    _like(dk_out, k, k.shape, "dk_out")
    if out is None:
        out = (torch.empty(q.shape, dtype=q.dtype, device=q.device), torch.empty(k.shape, dtype=k.dtype,
                                                                                device=k.device),
               None if q_weight is None else torch.empty_like(q_weight),
               None if k_weight is None else torch.empty_like(k_weight))
    else:
        _like(out[0], q, q.shape, "dq")
        _like(out[1], k, k.shape, "dk")
        for w, d, name in ((q_weight, out[2], "dq_weight"), (k_weight, out[3], "dk_weight")):
            if (w is None) != (d is None):
                raise ValueError(f"{name} goes with its weight: both or neither")
            if w is not None:
                _like(d, w, w.shape, name)
    dq, dk, dqw, dkw = out
    _keep, ws, n = _workspace(_b.tide_qk_norm_rope_grad_workspace(desc), workspace, q.device)
    _b.tide_qk_norm_rope_grad(desc, _heads(dq_out, "dq_out"), _heads(dk_out, "dk_out"),
                              _heads(q, "q") if q_weight is not None else None,
                              _heads(k, "k") if k_weight is not None else None, _heads(dq, "dq"), _heads(dk, "dk"),
                              0 if dqw is None else dqw.data_ptr(), 0 if dkw is None else dkw.data_ptr(), ws, n,
                              _stream(stream))
    return dq, dk, dqw, dkw


# ------------------------------------------------------------------ vocabulary head with cross entropy

def _ce_desc(x, weight, targets, ignore_index):
    if x.dtype != torch.bfloat16 or weight.dtype != torch.bfloat16:
        raise TypeError(f"x is {x.dtype} and weight {weight.dtype}: need bfloat16")
    _on_device(x, "x")
    if x.dim() != 2 or weight.dim() != 2 or x.shape[1] != weight.shape[1]:
        raise ValueError("need x [tokens, hidden] and weight [vocab, hidden]")
    for t, name in ((x, "x"), (weight, "weight")):
        if t.stride(1) != 1 and t.shape[1] > 1:
            raise ValueError(f"{name} has no contiguous last dimension")
    if targets.dtype not in _INT_BYTES or tuple(targets.shape) != (x.shape[0],):
        raise ValueError("targets must be an int32 or int64 tensor [tokens]")
    if targets.shape[0] > 1 and targets.stride(0) != 1:
        raise ValueError("targets must be contiguous")
    if weight.device != x.device or targets.device != x.device:
        raise ValueError("x, weight and targets must be on one device")
    return _b.CeDesc(x.shape[0], weight.shape[0], x.shape[1], x.data_ptr(), x.stride(0), weight.data_ptr(),
                     weight.stride(0), targets.data_ptr(), _INT_BYTES[targets.dtype], ignore_index)


def _per_token(t, x, name):
    if t.dtype != torch.float32 or t.device != x.device or tuple(t.shape) != (x.shape[0],) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor [tokens] on x's device")


def linear_cross_entropy(x, weight, targets, ignore_index: int = -100, out=None, workspace=None, stream=None):
    """(loss, lse), both fp32 [T]: every token's cross entropy of the logits ``x @ weight.T`` (x [T, H], weight
    [V, H], bf16) and the log of its sum of exponentials, which :func:`linear_cross_entropy_grad` takes.  The logits
    are not written to memory.  An ignored token's loss is 0."""
    desc = _ce_desc(x, weight, targets, ignore_index)
    if out is None:
        loss, lse = torch.empty((2, x.shape[0]), dtype=torch.float32, device=x.device)
    else:
        loss, lse = out
        _per_token(loss, x, "loss")
        _per_token(lse, x, "lse")
    _keep, ws, n = _workspace(_b.tide_ce_loss_workspace(desc), workspace, x.device)
    _b.tide_ce_loss(desc, loss.data_ptr(), lse.data_ptr(), ws, n, _stream(stream))
    return loss, lse


def linear_cross_entropy_grad(x, weight, targets, lse, dloss, ignore_index: int = -100, out=None, workspace=None,
                              stream=None):
    """(dx, dweight) of :func:`linear_cross_entropy` from its lse and the gradient ``dloss`` (fp32 [T]) of its losses
    (the mean over n tokens: 1 / n everywhere).  bf16, like x and weight."""
    desc = _ce_desc(x, weight, targets, ignore_index)
    _per_token(lse, x, "lse")
    _per_token(dloss, x, "dloss")
    if out is None:
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dw = torch.empty(weight.shape, dtype=weight.dtype, device=x.device)
    else:
        dx, dw = out
        _like(dx, x, x.shape, "dx")
        _like(dw, weight, weight.shape, "dweight")
    _keep, ws, n = _workspace(_b.tide_ce_grad_workspace(desc), workspace, x.device)
    _b.tide_ce_grad(desc, lse.data_ptr(), dloss.data_ptr(), dx.data_ptr(), dx.stride(0), dw.data_ptr(), dw.stride(0),
                    ws, n, _stream(stream))
    return dx, dw


# ------------------------------------------------------------------ SwiGLU with 8-bit checkpoints

class Ckpt8(NamedTuple):
    """Gate and up of a SwiGLU in 8 bits: e4m3 codes [rows, cols] (float8_e4m3fn, contiguous) and the biased
    exponents [rows, ceil(cols / 128)] (uint8) of their scales; value = code * 2^(exponent - 127)."""
    gate_codes: torch.Tensor
    gate_exps: torch.Tensor
    up_codes: torch.Tensor
    up_exps: torch.Tensor


def _ckpt_desc(ckpt, rows, cols, device):
    blocks = -(-cols // 128)
    for t, dt, w in ((ckpt[0], torch.float8_e4m3fn, cols), (ckpt[1], torch.uint8, blocks),
                     (ckpt[2], torch.float8_e4m3fn, cols), (ckpt[3], torch.uint8, blocks)):
        if t.dtype != dt or tuple(t.shape) != (rows, w) or not t.is_contiguous() or t.device != device:
            raise ValueError(f"a checkpoint tensor is {t.dtype} {tuple(t.shape)} on {t.device}: need contiguous {dt} "
                             f"({rows}, {w}) on {device}")
    return _b.Ckpt8Desc(*[t.data_ptr() for t in ckpt])


def new_ckpt8(rows: int, cols: int, device="cuda") -> Ckpt8:
    """An uninitialised checkpoint for [rows, cols]."""
    blocks = -(-cols // 128)
    make = lambda w, dt: torch.empty((rows, w), dtype=dt, device=device)  # noqa: E731
    return Ckpt8(make(cols, torch.float8_e4m3fn), make(blocks, torch.uint8), make(cols, torch.float8_e4m3fn),
                 make(blocks, torch.uint8))


def _rows(t, name):
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError(f"{name} must be [rows, cols] with contiguous rows")
    return t.stride(0)


def swiglu_ckpt8(gate, up, out=None, stream=None):
    """(h, ckpt): h = silu(gate) * up ([rows, cols], bf16 or fp32) and gate and up in 8 bits.  ``out = (h, ckpt)``."""
    dt = _dtype(gate, "gate")
    _on_device(gate, "gate")
    gs, us = _rows(gate, "gate"), _rows(up, "up")
    _like(up, gate, gate.shape, "up")
    rows, cols = gate.shape
    if out is None:
        h, ckpt = torch.empty((rows, cols), dtype=gate.dtype, device=gate.device), new_ckpt8(rows, cols, gate.device)
    else:
        h, ckpt = out
        _like(h, gate, gate.shape, "h")
    _b.tide_swiglu_ckpt8(rows, cols, dt, gate.data_ptr(), gs, up.data_ptr(), us, h.data_ptr(), _rows(h, "h"),
                         _ckpt_desc(ckpt, rows, cols, gate.device), _stream(stream))
    return h, ckpt


def swiglu_ckpt8_grad(ckpt: Ckpt8, dh, out=None, need_h: bool = True, stream=None):
    """(dgate, dup, h) of SwiGLU at the checkpoint's values; h, recomputed, is for the weight gradient of the
    projection that follows (None without ``need_h``).  ``out = (dgate, dup, h)``."""
    dt = _dtype(dh, "dh")
    _on_device(dh, "dh")
    ds = _rows(dh, "dh")
    rows, cols = dh.shape
    desc = _ckpt_desc(ckpt, rows, cols, dh.device)
    if out is None:
        out = [torch.empty((rows, cols), dtype=dh.dtype, device=dh.device) if i < 2 or need_h else None
               for i in range(3)]
    else:
        for t, name in zip(out, ("dgate", "dup", "h")):
            if t is not None:
                _like(t, dh, dh.shape, name)
    dgate, dup, h = out
    _b.tide_swiglu_ckpt8_grad(rows, cols, dt, desc, dh.data_ptr(), ds, dgate.data_ptr(), _rows(dgate, "dgate"),
                              dup.data_ptr(), _rows(dup, "dup"), 0 if h is None else h.data_ptr(),
                              0 if h is None else _rows(h, "h"), _stream(stream))
    return dgate, dup, h


def device_status(stream=None) -> int:
    """Reads and clears the operators' status word: TIDE_OK, or TIDE_ERR_TIMEOUT if a bounded wait expired."""
    return _b.tide_ops_device_status(_stream(stream))
