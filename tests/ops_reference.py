"""Plain 64-bit forms of the training-step operators, and bounds on what fp32
arithmetic may differ from them by.  Written from the formulas, independent of
the library and of the benchmark's plain forms; any torch device."""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24          # half an ulp of 1 in fp32
U16 = 2.0 ** -8           # bf16: twice the largest rounding error, relative
BLOCK = 128


def rounding(dtype) -> float:
    return U16 if dtype == torch.bfloat16 else 2 * U32


# ------------------------------------------------------------------ rotary table

def frequencies(R, base, scaling=None, factor=1.0, low=1.0, high=4.0, original=8192.0):
    out = []
    for i in range(R // 2):
        f = base ** (-2.0 * i / R)
        if scaling == "linear":
            f /= factor
        elif scaling == "by_parts":
            wave = 2 * math.pi / f
            if wave > original / low:
                f /= factor
            elif wave >= original / high:
                mix = (original / wave - low) / (high - low)
                f = (1 - mix) * f / factor + mix * f
        out.append(f)
    return torch.tensor(out, dtype=torch.float64)


# ------------------------------------------------------------------ head norm with rotation

def rotation(table, positions, D, interleaved):
    """[T, D, D] matrices that turn a head's columns at each token."""
    R = 0 if table is None else table.shape[1]
    T = positions.shape[0]
    M = torch.eye(D, dtype=torch.float64, device=positions.device).repeat(T, 1, 1)
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        c, s = table[positions, i].double(), table[positions, R // 2 + i].double()
        M[:, a, a], M[:, a, b] = c, -s
        M[:, b, a], M[:, b, b] = s, c
    return M


def qk_forward(x, w, M, eps):
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + eps) * w.double()
    return torch.einsum("tij,thj->thi", M, x)


def qk_backward(d, x, w, M, eps):
    """(dx, dw, sum of |terms| of dw)."""
    dy = torch.einsum("tji,thj->thi", M, d.double())
    if w is None:
        return dy, None, None
    x = x.double()
    D = x.shape[-1]
    r = 1 / torch.sqrt((x ** 2).mean(-1, keepdim=True) + eps)
    n = x * r
    g = dy * w.double()
    dx = r * (g - n * (g * n).sum(-1, keepdim=True) / D)
    return dx, (dy * n).sum((0, 1)), (dy * n).abs().sum((0, 1))


def qk_forward_bound(x, w, y, dtype, eps):
    """|error| of each element: the stored rounding, and the row's fp32 work (a chain of at most D/32 + 32
    roundings for the sum of squares, halved by the root, and a dozen after it) relative to its largest value."""
    D = x.shape[-1]
    top = x.double().abs()
    if w is not None:
        top = top / torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + eps) * w.double().abs()
    return rounding(dtype) * y.abs() + (D / 32 + 64) * U32 * 2 * top.amax(-1, keepdim=True)


def qk_backward_bound(d, x, w, M, dx, dtype, eps):
    D = x.shape[-1]
    top = d.double().abs().amax(-1, keepdim=True) * 2
    if w is not None:
        r = 1 / torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + eps)
        n = (x.double() * r).abs()
        top = top * w.double().abs().max()
        top = r * (top + n.amax(-1, keepdim=True) * top * n.mean(-1, keepdim=True))
    return rounding(dtype) * dx.abs() + (D / 32 + 96) * U32 * 2 * top


# ------------------------------------------------------------------ vocabulary cross entropy

def ce_logits(x, w):
    """(z, largest |error| of each z in fp32: every product and sum rounded or cut once)."""
    x, w = x.double(), w.double()
    return x @ w.t(), (x.shape[1] + 8) * 2 * U32 * (x.abs() @ w.abs().t())


def ce_loss(x, w, y, ignore=-100):
    """(loss, lse, bound on either's error)."""
    z, dz = ce_logits(x, w)
    lse = torch.logsumexp(z, 1)
    kept = y != ignore
    zy = z.gather(1, y.long().clamp(0, w.shape[0] - 1)[:, None])[:, 0]
    loss = torch.where(kept, lse - zy, torch.zeros_like(lse))
    # exponentials to 2^-20 relative, their sum in chains of at most 600, the logarithm, the difference
    return loss, lse, 2 * dz.amax(1) + 700 * U32 + 16 * U32 * (lse.abs() + zy.abs())


def ce_grad(x, w, y, lse, dloss, ignore=-100):
    """(dx, dw, bound of dx, bound of dw)."""
    z, ez = ce_logits(x, w)
    kept = (y != ignore)
    p = torch.exp(z - lse.double()[:, None])
    d = p.clone()
    at = torch.arange(len(y), device=y.device)
    d[at[kept], y.long()[kept]] -= 1.0
    scale = torch.where(kept, dloss.double(), torch.zeros_like(lse.double()))[:, None]
    d = d * scale
    # dz: its rounding to bf16, and p's error from z's, lse's and the exponential's
    ed = U16 * d.abs() + p * scale.abs() * (ez + 32 * U32 * (1 + z.abs() + lse.double().abs()[:, None]))
    x, w = x.double(), w.double()
    dx, dw = d @ w, d.t() @ x
    n = max(x.shape[0], w.shape[0]) + 64
    bx = ed @ w.abs() + n * 2 * U32 * (d.abs() @ w.abs()) + U16 * dx.abs()
    bw = ed.t() @ x.abs() + n * 2 * U32 * (d.abs().t() @ x.abs()) + U16 * dw.abs()
    return dx, dw, bx, bw


# ------------------------------------------------------------------ SwiGLU with 8-bit checkpoints

def e4m3_values():
    """The non-negative finite e4m3 values by code, from the format's definition."""
    out = []
    for c in range(127):
        e, m = c >> 3, c & 7
        out.append(m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return torch.tensor(out, dtype=torch.float64)


def pow2(exps):
    """2^(exps - 127) in 64 bits, exactly (from a table: a device's pow may be an ulp off)."""
    return torch.tensor([2.0 ** (k - 127) for k in range(256)], dtype=torch.float64, device=exps.device)[exps.long()]


def encode(x):
    """(value of each code [rows, cols] in 64 bits, exponents [rows, blocks]): the smallest e >= 1 with
    amax <= 448 * 2^(e - 127) over the finite values of a block, 127 for zeroes; values to the nearest code, ties to
    the even one; NaN for what is not finite."""
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    vals = e4m3_values().to(x.device)
    pad = torch.zeros((rows, blocks * BLOCK), dtype=torch.float64, device=x.device)
    pad[:, :cols] = x.double()
    pad = pad.view(rows, blocks, BLOCK)
    finite = torch.isfinite(pad)
    amax = torch.where(finite, pad.abs(), 0.0).amax(-1)
    exps = torch.full(amax.shape, 127, dtype=torch.int64, device=x.device)
    todo = amax > 0
    exps[todo] = 1
    for e in range(1, 248):
        exps = torch.where(todo & (amax > 448.0 * 2.0 ** (e - 127)), e + 1, exps)
    scale = pow2(exps)[..., None]
    mag = torch.where(finite, pad.abs(), 0.0) / scale
    hi = torch.searchsorted(vals, mag).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dlo, dhi = mag - vals[lo], vals[hi] - mag
    code = torch.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi)
    q = torch.where(finite, vals[code] * torch.sign(pad), float("nan"))
    return q.view(rows, blocks * BLOCK)[:, :cols], exps


def swiglu(g, u):
    g, u = g.double(), u.double()
    return g * torch.sigmoid(g) * u


def swiglu_grad(g, u, dh):
    g, u, dh = g.double(), u.double(), dh.double()
    s = torch.sigmoid(g)
    return dh * u * s * (1 + g * (1 - s)), dh * g * s, g * s * u


def swiglu_bound(exact, terms, g, dtype):
    """fp32: a dozen roundings of the product's terms, and exp(-g), whose argument is rounded; for bf16 the fast
    exponential and division (2^-21)."""
    fast = 8.0 if dtype == torch.bfloat16 else 1.0
    return rounding(dtype) * exact.abs() + (16 + 4 * g.double().abs().clamp(max=128)) * fast * U32 * terms.abs() + 1e-37
