"""Training-step operators on torch tensors: the compute next to the
collectives of an FSDP2 step.

Thin wrappers of the ``tide_*`` entry points of the same names
(``include/tide.h`` has the formulas): they check types and shapes, allocate
the outputs that are not passed in ``out`` and the scratch memory, and launch
on ``stream`` (default: the current stream).  Nothing is computed in Python.
A call with a ``stream`` is that call with the stream made current: what it
allocates, outputs and scratch memory, belongs to that stream, and is not
handed out again before the work on it is done.  A tensor that another stream
may still be using is the caller's to order, as with any asynchronous call.

Every operator has its gradient as a function of its own that takes and
returns plain tensors; gradients of parameters have the parameter's type and
can be written straight into a gradient arena with ``out``.  Where autograd
records and an input requires a gradient, an operator's outputs lead back to it
(``all_gather_gb300.autograd``), and ``out`` is refused, as torch's own
operators do; under ``torch.no_grad`` it is allowed.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _binding as _b

_DTYPES = {torch.bfloat16: _b.TIDE_DTYPE_BF16, torch.float32: _b.TIDE_DTYPE_F32}
_INT_BYTES = {torch.int32: 4, torch.int64: 8}
ROPE_SCALINGS = {None: 0, "linear": 1, "by_parts": 2}
_BF16, _F32 = torch.bfloat16, torch.float32
_raw_stream, _current_device, _empty = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice, torch.empty
_empty_like, _CONTIGUOUS = torch.empty_like, torch.contiguous_format
_recording = torch.is_grad_enabled

# These wrappers run once for every layer and token, in front of kernels of a
# few microseconds: each attribute is read once, checks are plain comparisons,
# and names that only an error needs are put together there.


def _stream() -> int:
    return _raw_stream(_current_device())


class _current:
    """Makes ``stream`` (a torch stream or a raw handle) the current one, which is the one that memory is allocated for."""

    def __init__(self, stream):
        raw = stream if isinstance(stream, int) else stream.cuda_stream
        self.other = None
        if raw != _stream():
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(raw) if raw > 1 else torch.cuda.default_stream()
            self.other = torch.cuda.stream(stream)

    def __enter__(self):
        if self.other is not None:
            self.other.__enter__()

    def __exit__(self, *error):
        if self.other is not None:
            self.other.__exit__(*error)


def _dtype(dtype, name):
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise TypeError(f"{name} is {dtype}: need bfloat16 or float32")
    return dt


def _device(t, name) -> int:
    """The current device, which is where a call launches: a tensor on another one is refused."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} is not on a CUDA device")
    if dev != _current_device():
        raise ValueError(f"{name} is on CUDA device {dev}, and device {_current_device()} is current")
    return dev


def _like(t, dtype, dev, shape, name):
    """Refuses a tensor that is not of this type, device and shape."""
    if t.dtype is not dtype or t.get_device() != dev:
        raise TypeError(f"{name} is {t.dtype} on {t.device}, expected {dtype} on CUDA device {dev}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _new(t):
    """A contiguous tensor like `t` (half the time of t.new_empty)."""
    return _empty_like(t, memory_format=_CONTIGUOUS)


def _scratch(n: int, workspace, like):
    """Scratch memory on the device of `like`: (tensor that keeps it alive, pointer, bytes)."""
    if workspace is None:
        workspace = _empty(n, dtype=torch.uint8, device=like.device)
        return workspace, workspace.data_ptr(), n
    if workspace.get_device() != like.get_device() or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the other tensors' device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _recorded(out, *inputs) -> bool:
    """Whether autograd has to know of this call."""
    if not _recording():
        return False
    for t in inputs:
        if t is not None and t.requires_grad:
            if out is not None:
                raise RuntimeError("out is given and an input requires a gradient: autograd cannot record this call")
            return True
    return False


def _written(*tensors):
    """Autograd's versions of tensors that the caller passed and the library has written."""
    for t in tensors:
        if t is not None and not t.is_inference():
            torch.autograd.graph.increment_version(t)


# ------------------------------------------------------------------ head norm with rotation

def rope_table(max_position: int, rotary_dim: int, base: float = 10000.0, scaling: Optional[str] = None,
               factor: float = 1.0, low_freq_factor: float = 1.0, high_freq_factor: float = 4.0,
               original: float = 8192.0, device=None, out=None, stream=None):
    """fp32 [max_position, rotary_dim]: cosines, then sines, of every position's angles.
    ``scaling``: None, "linear" (positions divided by ``factor``) or "by_parts"."""
    if stream is not None:
        with _current(stream):
            return rope_table(max_position, rotary_dim, base, scaling, factor, low_freq_factor, high_freq_factor, original,
                              device, out)
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling {scaling!r}: need one of {list(ROPE_SCALINGS)}")
    if out is None:
        out = _empty((max_position, rotary_dim), dtype=torch.float32, device="cuda" if device is None else device)
    elif (out.dtype != torch.float32 or not out.is_cuda or not out.is_contiguous()
          or tuple(out.shape) != (max_position, rotary_dim)):
        raise ValueError(f"out must be a contiguous float32 CUDA tensor [{max_position}, {rotary_dim}]")
    _device(out, "out")
    _b.tide_rope_table(max_position, rotary_dim, base, ROPE_SCALINGS[scaling], factor, low_freq_factor,
                       high_freq_factor, original, out.data_ptr(), _stream())
    return out


_packed_qk, _packed_heads, _packed_ckpt8 = _b.PackedCalls.qk, _b.PackedCalls.heads, _b.PackedCalls.ckpt8
_packed_attention, _packed_norm = _b.PackedCalls.attention, _b.PackedCalls.norm


def _heads(t, name):
    """A tensor of heads, with the dtype, device and shape already checked where it has to agree with another."""
    st = t.stride()
    if len(st) != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    if st[2] != 1 and t.shape[2] > 1:
        raise ValueError(f"{name} has no contiguous last dimension")
    return _packed_heads(t.data_ptr(), st[0], st[1])


def _qk_desc(q, k, table, positions, q_weight, k_weight, eps, interleaved):
    """(descriptor, device, q's shape, k's shape)."""
    dtype, dev, qs, ks = q.dtype, q.get_device(), q.shape, k.shape
    dt = _dtype(dtype, "q")
    if len(qs) != 3 or len(ks) != 3:
        raise ValueError("q and k must be [tokens, heads, head_dim]")
    T, Hq, D = qs
    if k.dtype is not dtype or k.get_device() != dev or ks[0] != T or ks[2] != D:
        raise ValueError("q and k must agree in type, device, tokens and head_dim")
    _device(q, "q")
    R = P = tp = pp = 0
    pos_bytes = 8
    if table is not None:
        if table.dtype is not _F32 or table.get_device() != dev or table.dim() != 2 or not table.is_contiguous():
            raise ValueError("table must be a contiguous float32 tensor [positions, rotary_dim] on q's device")
        P, R = table.shape
        pos_bytes = _INT_BYTES.get(positions.dtype, 0) if positions is not None else 0
        if not pos_bytes or positions.get_device() != dev:
            raise ValueError("positions must be an int32 or int64 tensor on q's device")
        if positions.shape != (T,) or not positions.is_contiguous():
            raise ValueError(f"positions must be contiguous of shape ({T},)")
        tp, pp = table.data_ptr(), positions.data_ptr()
    wq = wk = 0
    if q_weight is not None:
        _like(q_weight, dtype, dev, (D,), "q_weight")
        wq = q_weight.data_ptr()
    if k_weight is not None:
        _like(k_weight, dtype, dev, (D,), "k_weight")
        wk = k_weight.data_ptr()
    return _packed_qk(T, Hq, ks[1], D, R, P, tp, pp, pos_bytes, dt, 1 if interleaved else 0, eps, wq, wk), dev, qs, ks


def qk_norm_rope(q, k, table=None, positions=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                 interleaved: bool = False, out=None, stream=None):
    """(q_out, k_out): queries [T, Hq, D] and keys [T, Hk, D] normed for each head (where a weight [D] is given) and
    their first ``table.shape[1]`` columns rotated by the angles of ``positions`` [T] (where a table is given).
    ``out = (q_out, k_out)`` may be (q, k) themselves."""
    if stream is not None:
        with _current(stream):
            return qk_norm_rope(q, k, table, positions, q_weight, k_weight, eps, interleaved, out)
    if _recorded(out, q, k, table, q_weight, k_weight):
        from . import autograd
        return autograd.qk_norm_rope(q, k, table, positions, q_weight, k_weight, eps, interleaved)
    qh, kh = _heads(q, "q"), _heads(k, "k")
    desc, dev, qs, ks = _qk_desc(q, k, table, positions, q_weight, k_weight, eps, interleaved)
    if out is None:
        q_out, k_out = _new(q), _new(k)
    else:
        q_out, k_out = out
        _like(q_out, q.dtype, dev, qs, "q_out")
        _like(k_out, q.dtype, dev, ks, "k_out")
    status = _b.packed_calls().qk_norm_rope(desc, qh, kh, _heads(q_out, "q_out"), _heads(k_out, "k_out"),
                                            _stream())
    if status:
        _b._check(status, "tide_qk_norm_rope")
    if out is not None:
        _written(q_out, k_out)
    return q_out, k_out


def qk_norm_rope_grad(dq_out, dk_out, q, k, table=None, positions=None, q_weight=None, k_weight=None,
                      eps: float = 1e-6, interleaved: bool = False, out=None, workspace=None, stream=None):
    """(dq, dk, dq_weight, dk_weight) of :func:`qk_norm_rope` from its outputs' gradients and its inputs.  A weight
    that is None has no gradient (None), and its ``q`` or ``k`` is used for its shape only."""
    if stream is not None:
        with _current(stream):
            return qk_norm_rope_grad(dq_out, dk_out, q, k, table, positions, q_weight, k_weight, eps, interleaved, out,
                                     workspace)
    desc, dev, qs, ks = _qk_desc(q, k, table, positions, q_weight, k_weight, eps, interleaved)
    dtype = q.dtype
    _like(dq_out, dtype, dev, qs, "dq_out")
    _like(dk_out, dtype, dev, ks, "dk_out")
    if out is None:
        dq, dk = _new(q), _new(k)
        dqw = None if q_weight is None else _new(q_weight)
        dkw = None if k_weight is None else _new(k_weight)
    else:
        dq, dk, dqw, dkw = out
        _like(dq, dtype, dev, qs, "dq")
        _like(dk, dtype, dev, ks, "dk")
        for w, d, name in ((q_weight, dqw, "dq_weight"), (k_weight, dkw, "dk_weight")):
            if (w is None) != (d is None):
                raise ValueError(f"{name} goes with its weight: both or neither")
            if w is not None:
                _like(d, dtype, dev, (qs[2],), name)
    lib, ws, n = _b.packed_calls(), 0, 0
    if q_weight is not None or k_weight is not None or workspace is not None:
        need = _b._size(lib.qk_norm_rope_grad_workspace(desc), "tide_qk_norm_rope_grad_workspace")
        _keep, ws, n = _scratch(need, workspace, q)
    status = lib.qk_norm_rope_grad(desc, _heads(dq_out, "dq_out"), _heads(dk_out, "dk_out"),
                                   None if q_weight is None else _heads(q, "q"),
                                   None if k_weight is None else _heads(k, "k"), _heads(dq, "dq"), _heads(dk, "dk"),
                                   0 if dqw is None else dqw.data_ptr(), 0 if dkw is None else dkw.data_ptr(), ws, n,
                                   _stream())
    if status:
        _b._check(status, "tide_qk_norm_rope_grad")
    if out is not None:
        _written(dq, dk, dqw, dkw)
    return dq, dk, dqw, dkw


# ------------------------------------------------------------------ vocabulary head with cross entropy

def _ce_desc(x, weight, targets, ignore_index):
    """(descriptor, device, tokens)."""
    if x.dtype is not _BF16 or weight.dtype is not _BF16:
        raise TypeError(f"x is {x.dtype} and weight {weight.dtype}: need bfloat16")
    dev, xs, ws = _device(x, "x"), x.shape, weight.shape
    if len(xs) != 2 or len(ws) != 2 or xs[1] != ws[1]:
        raise ValueError("need x [tokens, hidden] and weight [vocab, hidden]")
    T, H = xs
    xt, wt = x.stride(), weight.stride()
    if H > 1 and (xt[1] != 1 or wt[1] != 1):
        raise ValueError("x or weight has no contiguous last dimension")
    target_bytes = _INT_BYTES.get(targets.dtype)
    if target_bytes is None or targets.shape != (T,) or not targets.is_contiguous():
        raise ValueError("targets must be a contiguous int32 or int64 tensor [tokens]")
    if weight.get_device() != dev or targets.get_device() != dev:
        raise ValueError("x, weight and targets must be on one device")
    return _b.CeDesc(T, ws[0], H, x.data_ptr(), xt[0], weight.data_ptr(), wt[0], targets.data_ptr(), target_bytes,
                     ignore_index), dev, T


def _per_token(t, dev, T, name):
    if t.dtype is not _F32 or t.get_device() != dev or t.shape != (T,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor [tokens] on x's device")


def _rows(t, name) -> int:
    """Row stride of a matrix with contiguous rows."""
    st = t.stride()
    if len(st) != 2 or (st[1] != 1 and t.shape[1] > 1):
        raise ValueError(f"{name} must be [rows, cols] with contiguous rows")
    return st[0]


def linear_cross_entropy(x, weight, targets, ignore_index: int = -100, out=None, workspace=None, stream=None):
    """(loss, lse), both fp32 [T]: every token's cross entropy of the logits ``x @ weight.T`` (x [T, H], weight
    [V, H], bf16) and the log of its sum of exponentials, which :func:`linear_cross_entropy_grad` takes.  The logits
    are not written to memory.  An ignored token's loss is 0.  lse itself has no gradient."""
    if stream is not None:
        with _current(stream):
            return linear_cross_entropy(x, weight, targets, ignore_index, out, workspace)
    if _recorded(out, x, weight):
        from . import autograd
        return autograd.loss_and_lse(x, weight, targets, ignore_index, workspace)
    desc, dev, T = _ce_desc(x, weight, targets, ignore_index)
    if out is None:
        loss, lse = _empty(T, dtype=_F32, device=x.device), _empty(T, dtype=_F32, device=x.device)
    else:
        loss, lse = out
        _per_token(loss, dev, T, "loss")
        _per_token(lse, dev, T, "lse")
    _keep, ws, n = _scratch(_b.tide_ce_loss_workspace(desc), workspace, x)
    _b.tide_ce_loss(desc, loss.data_ptr(), lse.data_ptr(), ws, n, _stream())
    if out is not None:
        _written(loss, lse)
    return loss, lse


def linear_cross_entropy_grad(x, weight, targets, lse, dloss, ignore_index: int = -100, out=None, workspace=None,
                              stream=None):
    """(dx, dweight) of :func:`linear_cross_entropy` from its lse and the gradient ``dloss`` (fp32 [T]) of its losses
    (the mean over n tokens: 1 / n everywhere).  bf16, like x and weight."""
    if stream is not None:
        with _current(stream):
            return linear_cross_entropy_grad(x, weight, targets, lse, dloss, ignore_index, out, workspace)
    desc, dev, T = _ce_desc(x, weight, targets, ignore_index)
    _per_token(lse, dev, T, "lse")
    _per_token(dloss, dev, T, "dloss")
    if out is None:
        dx, dw = _new(x), _new(weight)
    else:
        dx, dw = out
        _like(dx, _BF16, dev, x.shape, "dx")
        _like(dw, _BF16, dev, weight.shape, "dweight")
    _keep, ws, n = _scratch(_b.tide_ce_grad_workspace(desc), workspace, x)
    _b.tide_ce_grad(desc, lse.data_ptr(), dloss.data_ptr(), dx.data_ptr(), _rows(dx, "dx"), dw.data_ptr(),
                    _rows(dw, "dweight"), ws, n, _stream())
    if out is not None:
        _written(dx, dw)
    return dx, dw


# ------------------------------------------------------------------ SwiGLU with 8-bit checkpoints

class Ckpt8(NamedTuple):
    """Gate and up of a SwiGLU in 8 bits: e4m3 codes [rows, cols] (float8_e4m3fn, contiguous) and the biased
    exponents [rows, ceil(cols / 128)] (uint8) of their scales; value = code * 2^(exponent - 127)."""
    gate_codes: torch.Tensor
    gate_exps: torch.Tensor
    up_codes: torch.Tensor
    up_exps: torch.Tensor


_E4M3, _U8 = torch.float8_e4m3fn, torch.uint8


def _ckpt_desc(ckpt, rows, cols, dev):
    codes, exps = (rows, cols), (rows, -(-cols // 128))
    g8, ge, u8, ue = ckpt
    for t, dt, shape in ((g8, _E4M3, codes), (ge, _U8, exps), (u8, _E4M3, codes), (ue, _U8, exps)):
        if t.dtype is not dt or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
            raise ValueError(f"a checkpoint tensor is {t.dtype} {tuple(t.shape)} on {t.device}: need contiguous {dt} "
                             f"{shape} on CUDA device {dev}")
    return _packed_ckpt8(g8.data_ptr(), ge.data_ptr(), u8.data_ptr(), ue.data_ptr())


def new_ckpt8(rows: int, cols: int, device="cuda") -> Ckpt8:
    """An uninitialised checkpoint for [rows, cols]."""
    codes, exps = (rows, cols), (rows, -(-cols // 128))
    return Ckpt8(_empty(codes, dtype=_E4M3, device=device), _empty(exps, dtype=_U8, device=device),
                 _empty(codes, dtype=_E4M3, device=device), _empty(exps, dtype=_U8, device=device))


def swiglu_ckpt8(gate, up, out=None, stream=None):
    """(h, ckpt): h = silu(gate) * up ([rows, cols], bf16 or fp32) and gate and up in 8 bits.  ``out = (h, ckpt)``."""
    if stream is not None:
        with _current(stream):
            return swiglu_ckpt8(gate, up, out)
    if _recorded(out, gate, up):
        from . import autograd
        return autograd.swiglu_and_ckpt8(gate, up)
    dtype, shape = gate.dtype, gate.shape
    dt = _dtype(dtype, "gate")
    dev = _device(gate, "gate")
    gs, us = _rows(gate, "gate"), _rows(up, "up")
    _like(up, dtype, dev, shape, "up")
    rows, cols = shape
    if out is None:
        device = gate.device
        h, ckpt, hs = _new(gate), new_ckpt8(rows, cols, device), cols
        desc = _packed_ckpt8(*[t.data_ptr() for t in ckpt])
    else:
        h, ckpt = out
        _like(h, dtype, dev, shape, "h")
        hs, desc = _rows(h, "h"), _ckpt_desc(ckpt, rows, cols, dev)
    status = _b.packed_calls().swiglu_ckpt8(rows, cols, dt, gate.data_ptr(), gs, up.data_ptr(), us, h.data_ptr(), hs,
                                            desc, _stream())
    if status:
        _b._check(status, "tide_swiglu_ckpt8")
    if out is not None:
        _written(h, *ckpt)
    return h, ckpt


def swiglu_ckpt8_grad(ckpt: Ckpt8, dh, out=None, need_h: bool = True, stream=None):
    """(dgate, dup, h) of SwiGLU at the checkpoint's values; h, recomputed, is for the weight gradient of the
    projection that follows (None without ``need_h``).  ``out = (dgate, dup, h)``."""
    if stream is not None:
        with _current(stream):
            return swiglu_ckpt8_grad(ckpt, dh, out, need_h)
    dtype, shape = dh.dtype, dh.shape
    dt = _dtype(dtype, "dh")
    dev = _device(dh, "dh")
    ds = _rows(dh, "dh")
    rows, cols = shape
    desc = _ckpt_desc(ckpt, rows, cols, dev)
    if out is None:
        dgate, dup = _new(dh), _new(dh)
        h = _new(dh) if need_h else None
    else:
        dgate, dup, h = out
        for t, name in ((dgate, "dgate"), (dup, "dup"), (h, "h")):
            if t is not None:
                _like(t, dtype, dev, shape, name)
    status = _b.packed_calls().swiglu_ckpt8_grad(rows, cols, dt, desc, dh.data_ptr(), ds, dgate.data_ptr(),
                                                 _rows(dgate, "dgate"), dup.data_ptr(), _rows(dup, "dup"),
                                                 0 if h is None else h.data_ptr(), 0 if h is None else _rows(h, "h"),
                                                 _stream())
    if status:
        _b._check(status, "tide_swiglu_ckpt8_grad")
    if out is not None:
        _written(dgate, dup, h)
    return dgate, dup, h


# ------------------------------------------------------------------ attention over packed sequences

def _attention_desc(q, k, v, offsets, causal, scale):
    """(descriptor, device, q's shape)."""
    dtype, dev, qs, ks = q.dtype, q.get_device(), q.shape, k.shape
    if dtype is not _BF16:
        raise TypeError(f"q is {dtype}: need bfloat16")
    if len(qs) != 3 or len(ks) != 3:
        raise ValueError("q, k and v must be [tokens, heads, head_dim]")
    T, Hq, D = qs
    if (k.dtype is not dtype or v.dtype is not dtype or k.get_device() != dev or v.get_device() != dev or ks[0] != T
            or ks[2] != D or v.shape != ks):
        raise ValueError("q, k and v must agree in type, device, tokens and head_dim, k and v in heads")
    _device(q, "q")
    n = op = 0
    nbytes = 8
    if offsets is not None:
        nbytes = _INT_BYTES.get(offsets.dtype)
        if (nbytes is None or offsets.get_device() != dev or offsets.dim() != 1 or not offsets.is_contiguous()
                or not offsets.shape[0]):
            raise ValueError("offsets must be a contiguous int32 or int64 tensor [sequences + 1] on q's device")
        n, op = offsets.shape[0] - 1, offsets.data_ptr()
    if scale is None:
        scale = D ** -0.5 if D else 1.0
    return _packed_attention(T, Hq, ks[1], D, 1 if causal else 0, scale, nbytes, n, op, 0), dev, qs


def _lse(t, dev, qs):
    if t.dtype is not _F32 or t.get_device() != dev or t.shape != (qs[1], qs[0]) or not t.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 tensor [{qs[1]}, {qs[0]}] on q's device")


def attention(q, k, v, offsets=None, causal: bool = True, scale: Optional[float] = None, out=None, stream=None):
    """(o, lse): softmax attention of q [T, Hq, D] over k and v [T, Hk, D] (bf16; query head h reads key head
    h * Hk // Hq), and the log of every row's sum of exponentials, fp32 [Hq, T], which :func:`attention_grad` takes.
    ``offsets`` (int32 or int64 [n + 1], on the device): sequence i is the tokens offsets[i] to offsets[i + 1] - 1, and
    sees itself only; without them all tokens are one sequence.  ``causal``: a token sees no later one.  ``scale`` of
    the scores: default 1 / sqrt(D).  A token of no sequence gets 0 (lse: -inf).  lse itself has no gradient."""
    if stream is not None:
        with _current(stream):
            return attention(q, k, v, offsets, causal, scale, out)
    if _recorded(out, q, k, v):
        from . import autograd
        return autograd.attention_and_lse(q, k, v, offsets, causal, scale)
    desc, dev, qs = _attention_desc(q, k, v, offsets, causal, scale)
    if out is None:
        o, lse = _new(q), _empty((qs[1], qs[0]), dtype=_F32, device=q.device)
    else:
        o, lse = out
        _like(o, _BF16, dev, qs, "o")
        _lse(lse, dev, qs)
    status = _b.packed_calls().attention_forward(desc, _heads(q, "q"), _heads(k, "k"), _heads(v, "v"), _heads(o, "o"),
                                                 lse.data_ptr(), _stream())
    if status:
        _b._check(status, "tide_attention")
    if out is not None:
        _written(o, lse)
    return o, lse


def attention_grad(do, q, k, v, o, lse, offsets=None, causal: bool = True, scale: Optional[float] = None, out=None,
                   workspace=None, stream=None):
    """(dq, dk, dv) of :func:`attention` from the gradient ``do`` of its o, its inputs, and its outputs o and lse."""
    if stream is not None:
        with _current(stream):
            return attention_grad(do, q, k, v, o, lse, offsets, causal, scale, out, workspace)
    desc, dev, qs = _attention_desc(q, k, v, offsets, causal, scale)
    _like(do, _BF16, dev, qs, "do")
    _like(o, _BF16, dev, qs, "o")
    _lse(lse, dev, qs)
    if out is None:
        dq, dk, dv = _new(q), _new(k), _new(v)
    else:
        dq, dk, dv = out
        _like(dq, _BF16, dev, qs, "dq")
        _like(dk, _BF16, dev, k.shape, "dk")
        _like(dv, _BF16, dev, k.shape, "dv")
    lib = _b.packed_calls()
    need = _b._size(lib.attention_grad_workspace(desc), "tide_attention_grad_workspace")
    _keep, ws, n = _scratch(need, workspace, q)
    status = lib.attention_grad(desc, _heads(do, "do"), _heads(q, "q"), _heads(k, "k"), _heads(v, "v"), _heads(o, "o"),
                                lse.data_ptr(), _heads(dq, "dq"), _heads(dk, "dk"), _heads(dv, "dv"), ws, n, _stream())
    if status:
        _b._check(status, "tide_attention_grad")
    if out is not None:
        _written(dq, dk, dv)
    return dq, dk, dv


# ------------------------------------------------------------------ layer norm

def _norm_desc(x, weight, bias, eps, center):
    """(descriptor, device, x's shape)."""
    dtype, shape = x.dtype, x.shape
    dt = _dtype(dtype, "x")
    dev = _device(x, "x")
    if len(shape) != 2:
        raise ValueError("x must be [rows, cols]")
    wp = bp = 0
    if weight is not None:
        _like(weight, dtype, dev, shape[1:], "weight")
        wp = _vector(weight, "weight")
    if bias is not None:
        _like(bias, dtype, dev, shape[1:], "bias")
        bp = _vector(bias, "bias")
    return _packed_norm(shape[0], shape[1], dt, 1 if center else 0, wp, bp, eps), dev, shape


def _vector(t, name) -> int:
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, center: bool = True, out=None, stream=None):
    """Every row of x [rows, cols] (bf16 or fp32) less its mean, over the root of its variance plus ``eps``, times
    ``weight`` plus ``bias`` [cols] (where given).  ``center=False``: the mean is not taken off, which is the
    root-mean-square norm.  ``out`` may be x itself."""
    if stream is not None:
        with _current(stream):
            return layer_norm(x, weight, bias, eps, center, out)
    if _recorded(out, x, weight, bias):
        from . import autograd
        return autograd.layer_norm(x, weight, bias, eps, center)
    desc, dev, shape = _norm_desc(x, weight, bias, eps, center)
    if out is None:
        y = _new(x)
    else:
        y = out
        _like(y, x.dtype, dev, shape, "out")
    status = _b.packed_calls().layer_norm(desc, x.data_ptr(), _rows(x, "x"), y.data_ptr(), _rows(y, "out"), _stream())
    if status:
        _b._check(status, "tide_layer_norm")
    if out is not None:
        _written(y)
    return y


def layer_norm_grad(dy, x, weight=None, bias=None, eps: float = 1e-5, center: bool = True, out=None, workspace=None,
                    stream=None):
    """(dx, dweight, dbias) of :func:`layer_norm` from its output's gradient and its inputs; a weight or bias that is
    None has no gradient (None).  ``out = (dx, dweight, dbias)``, of which dx may be dy or x."""
    if stream is not None:
        with _current(stream):
            return layer_norm_grad(dy, x, weight, bias, eps, center, out, workspace)
    desc, dev, shape = _norm_desc(x, weight, bias, eps, center)
    dtype = x.dtype
    _like(dy, dtype, dev, shape, "dy")
    if out is None:
        dx = _new(x)
        dw = None if weight is None else _new(weight)
        db = None if bias is None else _new(bias)
    else:
        dx, dw, db = out
        _like(dx, dtype, dev, shape, "dx")
        for w, d, name in ((weight, dw, "dweight"), (bias, db, "dbias")):
            if (w is None) != (d is None):
                raise ValueError(f"{name} goes with its parameter: both or neither")
            if w is not None:
                _like(d, dtype, dev, shape[1:], name)
    lib, ws, n = _b.packed_calls(), 0, 0
    if weight is not None or bias is not None:
        need = _b._size(lib.layer_norm_grad_workspace(desc), "tide_layer_norm_grad_workspace")
        _keep, ws, n = _scratch(need, workspace, x)
    status = lib.layer_norm_grad(desc, dy.data_ptr(), _rows(dy, "dy"), x.data_ptr(), _rows(x, "x"), dx.data_ptr(),
                                 _rows(dx, "dx"), 0 if dw is None else _vector(dw, "dweight"),
                                 0 if db is None else _vector(db, "dbias"), ws, n, _stream())
    if status:
        _b._check(status, "tide_layer_norm_grad")
    if out is not None:
        _written(dx, dw, db)
    return dx, dw, db


def device_status(stream=None) -> int:
    """Reads and clears the operators' status word: TIDE_OK, or TIDE_ERR_TIMEOUT if a bounded wait expired."""
    if stream is not None:
        with _current(stream):
            return device_status()
    return _b.tide_ops_device_status(_stream())
