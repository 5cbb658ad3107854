"""Plain 64-bit forms of attention over packed sequences and of layer norm, and bounds on what the kernels' arithmetic
may differ from them by.  Written from the formulas, independent of the library and of the benchmark's plain forms; any
torch device."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24   # half a step of fp32, relative
U16 = 2.0 ** -8    # half a step of bf16, relative
CUT = 2.0 ** -23   # a step of fp32: the tensor cores cut their sums
TINY = 2.0 ** -126  # exponentials below it are 0


def rounding(dtype) -> float:
    return U16 if dtype == torch.bfloat16 else U32


# ------------------------------------------------------------------ attention

def sequence_of(offsets, T):
    """Number of every token's sequence, -1 for none."""
    seq = [-1] * T
    for i, (a, b) in enumerate(zip(offsets, offsets[1:])):
        for t in range(max(a, 0), min(b, T)):
            seq[t] = i
    return torch.tensor(seq)


def visible(offsets, T, causal, device):
    """[T, T]: whether row r sees key c."""
    seq = torch.zeros(T, dtype=torch.long) if offsets is None else sequence_of(offsets, T)
    see = (seq[:, None] == seq[None, :]) & (seq[:, None] >= 0)
    if causal:
        see &= torch.ones(T, T, dtype=torch.bool).tril()
    return see.to(device)


class Attention:
    """All values of a small problem, [Hq, T, ...] in 64 bits; what a row does not see takes no part in it."""

    def __init__(self, q, k, v, offsets=None, causal=True, scale=None):
        T, Hq, D = q.shape
        self.group = Hq // k.shape[1]
        self.scale = D ** -0.5 if scale is None else scale
        self.see = visible(offsets, T, causal, q.device)
        self.q = q.double().permute(1, 0, 2)
        self.k, self.v = (x.double().repeat_interleave(self.group, 1).permute(1, 0, 2) for x in (k, v))
        # products row by row over what is seen: 0 times a NaN that is not seen would be one
        self.kc, self.vc = (torch.where(torch.isfinite(x), x, 0.0) for x in (self.k, self.v))
        self.s = torch.where(self.see, self.scale * (self.q @ self.k.transpose(1, 2)), -torch.inf)
        self.some = self.see.any(1)
        self.lse = torch.logsumexp(self.s, 2)
        self.p = torch.where(self.see, torch.exp(self.s - self.lse[..., None]), 0.0)
        self.o = self.seen(self.p, self.v)
        # scores: products of two bf16 are whole in fp32, their sum is cut at every step; then two roundings more
        self.ds_score = self.scale * (self.q.abs() @ self.k.abs().transpose(1, 2)) * (D + 8) * CUT
        self.D, self.n = D, int(self.see.sum(1).max())

    def seen(self, p, x, see=None):
        """p @ x over the pairs that are seen; p is 0 elsewhere."""
        see = self.see if see is None else see
        out = p @ torch.where(torch.isfinite(x), x, 0.0)
        bad = ~torch.isfinite(x)
        if bad.any():
            hit = see.double() @ bad.double() > 0
            out = torch.where(hit, torch.nan, out)
        return out

    def tokens(self, x):
        return x.permute(1, 0, 2)

    def keys(self, x):
        """Sums over the query heads of a key head, [T, Hk, D]."""
        return x.reshape(-1, self.group, *x.shape[1:]).sum(1).permute(1, 0, 2)

    def p_error(self):
        """Relative error of a p before its rounding to bf16: the scores', and the exponential's and maximum's few steps
        of what is exponentiated."""
        size = torch.where(self.see, self.s.abs() + self.lse.abs()[..., None], 0.0)
        return torch.where(self.see, self.ds_score, 0.0) + 8 * U32 * (1 + size)

    def o_bound(self):
        e = self.p_error().amax(2, keepdim=True)
        size = self.p @ self.vc.abs() + TINY * (self.see.double() @ self.vc.abs())
        return self.tokens((U16 + 2 * e + (self.n + 16) * CUT) * size + U16 * self.o.abs() + 1e-37)

    def lse_bound(self):
        return self.p_error().amax(2) + (self.n + 16) * U32 + 4 * U32 * self.lse.abs()

    def grads(self, do, o, lse):
        """(dq, dk, dv) from the o and lse that the operator takes, and their bounds."""
        do = do.double().permute(1, 0, 2)
        o, lse = o.double().permute(1, 0, 2), lse.double()
        p = torch.where(self.see, torch.exp(self.s - lse[..., None]), 0.0)
        dp = do @ self.v.transpose(1, 2)
        delta = (do * o).sum(2)
        ds = torch.where(self.see, p * (dp - delta[..., None]), 0.0)
        seen_by = self.see.t()
        dv = self.keys(self.seen(p.transpose(1, 2), do, seen_by))
        dq = self.tokens(self.scale * self.seen(ds, self.k))
        dk = self.keys(self.scale * self.seen(ds.transpose(1, 2), self.q, seen_by))
        fin = lambda x: torch.where(torch.isfinite(x), x, 0.0)  # noqa: E731
        e = self.p_error()
        long = (self.n * self.group + 16) * CUT
        ddp = (do.abs() @ self.vc.abs().transpose(1, 2) + (do.abs() * o.abs()).sum(2)[..., None]) * (self.D + 8) * CUT
        dds = torch.where(self.see, fin(p * ddp + (U16 + 2 * e) * ds.abs() + TINY * (dp - delta[..., None]).abs()), 0.0)
        dpp = torch.where(self.see, fin((U16 + 2 * e) * p) + TINY, 0.0)
        dsa, pa = fin(ds.abs()), fin(p)
        bq = self.tokens(self.scale * ((dds + long * dsa) @ self.kc.abs())) + U16 * dq.abs() + 1e-37
        bk = self.keys(self.scale * ((dds + long * dsa).transpose(1, 2) @ fin(self.q).abs())) + U16 * dk.abs() + 1e-37
        bv = self.keys((dpp + long * pa).transpose(1, 2) @ fin(do).abs()) + U16 * dv.abs() + 1e-37
        return (dq, dk, dv), (bq, bk, bv)


# ------------------------------------------------------------------ layer norm

class Norm:
    """Layer norm of x [rows, cols] and its gradient."""

    def __init__(self, x, w, b, eps, center):
        self.x = x.double()
        self.C = x.shape[1]
        self.w = None if w is None else w.double()
        self.b = None if b is None else b.double()
        self.center, self.dtype = center, x.dtype
        self.mean = self.x.mean(1, keepdim=True) if center else torch.zeros_like(self.x[:, :1])
        self.r = 1 / torch.sqrt(((self.x - self.mean) ** 2).mean(1, keepdim=True) + eps)
        self.n = (self.x - self.mean) * self.r
        y = self.n if w is None else self.n * self.w
        self.y = y if b is None else y + self.b
        # a sum over a row: 32 elements a thread, five exchanges, up to 32 warps
        self.chain = 72 * U32
        # error of n: the mean's (a sum's, of values as large as the largest), relative to the row's spread, and r's
        top = self.x.abs().amax(1, keepdim=True)
        self.dn = (self.chain * top * self.r if center else 0) * (1 + self.n.abs()) + (self.chain + 6 * U32) * self.n.abs()

    def bound(self):
        w = 1 if self.w is None else self.w.abs()
        size = self.n.abs() * w + (0 if self.b is None else self.b.abs())
        return w * self.dn + 3 * U32 * size + rounding(self.dtype) * self.y.abs() + 1e-44

    def grads(self, dy):
        dy = dy.double()
        g = dy if self.w is None else dy * self.w
        along = (g * self.n).mean(1, keepdim=True)
        level = g.mean(1, keepdim=True) if self.center else 0
        dx = self.r * (g - level - self.n * along)
        ga = g.abs()
        d_along = ((ga * (self.dn + 2 * self.chain * self.n.abs())).mean(1, keepdim=True))
        d_level = self.chain * ga.mean(1, keepdim=True) if self.center else 0
        err = self.r * (self.n.abs() * d_along + self.dn * along.abs() + d_level +
                        8 * U32 * (ga + abs(level) + (self.n * along).abs()))
        err = err + (self.chain + 6 * U32 + (self.dn.mean(1, keepdim=True))) * dx.abs()
        rows = self.x.shape[0]
        long = (rows + 64) * U32
        dw = (dy * self.n).sum(0)
        bw = (dy.abs() * (self.dn + long * self.n.abs())).sum(0) + rounding(self.dtype) * dw.abs() + 1e-44
        db = dy.sum(0)
        bb = long * dy.abs().sum(0) + rounding(self.dtype) * db.abs() + 1e-44
        return (dx, dw, db), (err + rounding(self.dtype) * dx.abs() + 1e-44, bw, bb)
