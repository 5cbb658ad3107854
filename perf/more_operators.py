"""Cases, inputs and plain forms of attention over packed sequences and of layer norm, for measuring them.

Two operators, each in both directions:

* ``attn``   softmax attention of whole prompts: causal or not, grouped heads, sequences of several lengths in one batch
* ``norm``   layer norm (or, without its centre, root-mean-square norm) of rows, with weight and bias

``own`` selects between the plain form (elementary torch operations in fp32, rounded once at the end) and the
framework's entry points.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ---------------------------------------------------------------------------------------------------- cases

def _attn(op, T, Hq, Hk, D, sequences=1, split=0, tail=0, causal=True, packed=True):
    """`sequences` of lengths drawn from `split` share the first T - tail tokens; the tail belongs to none."""
    return dict(op=op, T=T, Hq=Hq, Hk=Hk, D=D, sequences=sequences, split=split, tail=tail, causal=causal, packed=packed,
                dtype="bf16")


def _norm(op, T, C, weight=True, bias=True, center=True, dtype="bf16"):
    return dict(op=op, T=T, C=C, weight=weight, bias=bias, center=center, dtype=dtype)


def listed():
    return [
        # one short prompt of a mixture-of-experts layer with 32 query and 4 key heads: what the call itself costs
        dict(name="attn_fwd_short", **_attn("attn_fwd", 61, 32, 4, 128)),
        # many short documents, heads of an odd size and number
        dict(name="attn_fwd_many", **_attn("attn_fwd", 4099, 7, 1, 80, sequences=97, split=5, packed=False)),
        # a training micro-batch of documents packed into one row, its padding behind them
        dict(name="attn_fwd_packed", **_attn("attn_fwd", 16384, 32, 4, 128, sequences=9, split=1, tail=100)),
        # one long document, 32 query and 8 key heads
        dict(name="attn_fwd_8k", **_attn("attn_fwd", 8192, 32, 8, 128)),
        # a diffusion transformer's block: 40 heads, every token sees every other, an odd number of them
        dict(name="attn_fwd_full", **_attn("attn_fwd", 4681, 40, 40, 128, causal=False)),
        # a few short documents on the way back, heads of 64
        dict(name="attn_bwd_short", **_attn("attn_bwd", 203, 8, 2, 64, sequences=3, split=2)),
        # the packed micro-batch on the way back
        dict(name="attn_bwd_packed", **_attn("attn_bwd", 8192, 32, 4, 128, sequences=7, split=3, tail=77)),
        # the long document on the way back
        dict(name="attn_bwd_8k", **_attn("attn_bwd", 8192, 32, 8, 128)),
        # one token of a generation step
        dict(name="norm_fwd_one_token", **_norm("norm_fwd", 1, 5120)),
        # a training micro-batch in front of a decoder layer: weight only, not centred
        dict(name="norm_fwd_32k", **_norm("norm_fwd", 32768, 4096, bias=False, center=False)),
        # odd rows and columns, fp32
        dict(name="norm_bwd_ragged_f32", **_norm("norm_bwd", 1003, 1001, dtype="f32")),
        # a training micro-batch of a diffusion transformer on the way back
        dict(name="norm_bwd_32k", **_norm("norm_bwd", 32768, 5120)),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attn_fwd", "attn_fwd", "attn_bwd", "attn_bwd", "norm_fwd", "norm_bwd"))
    if op.startswith("attn"):
        D = rng.choice((64, 80, 96, 112, 128, 128, 128))
        Hk = rng.choice((1, 2, 4, 5, 8))
        Hq = Hk * rng.choice((1, 2, 4, 7, 8))
        T = min(_log(rng, 1, 8192), int(math.sqrt(8192 * 8192 * 32 / Hq)))
        causal = rng.random() < 0.75
        if not causal:
            T = min(T, int(8192 * math.sqrt(16 / max(16, Hq))))
        tail = rng.choice((0, 0, 0, _log(rng, 1, 128)))
        return _attn(op, T, Hq, Hk, D, sequences=rng.choice((1, 1, 2, _log(rng, 1, 64))), split=rng.randrange(1 << 20),
                     tail=min(tail, T - 1), causal=causal, packed=rng.random() < 0.5)
    dtype = rng.choice(("bf16", "bf16", "f32"))
    step = rng.choice((256, 64, 8, 1))
    C = step * ((_log(rng, 64, 16384) // step - 1) | 1) if step < 64 else step * max(1, _log(rng, 64, 16384) // step)
    T = min(_log(rng, 1, 65536), (32768 if dtype == "bf16" else 16384) * 4096 // C)
    weight = rng.random() < 0.9
    return _norm(op, T, C, weight=weight, bias=weight and rng.random() < 0.5, center=rng.random() < 0.6, dtype=dtype)


def _bounds(c):
    """Where the sequences begin, and where the last one ends."""
    n = c["T"] - c["tail"]
    rng = random.Random(c["split"])
    return [0] + sorted(rng.randint(0, n) for _ in range(c["sequences"] - 1)) + [n]


# --------------------------------------------------------------------------------------------------- inputs

def _normal(g, shape, scale=1.0, dtype=torch.float32):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return x.mul_(scale).to(dtype)


def _prepare_attn(c, g):
    dt, T, Hq, Hk, D = DTYPES[c["dtype"]], c["T"], c["Hq"], c["Hk"], c["D"]
    if c["packed"]:  # views of the packed q, k, v projection's output
        qkv = _normal(g, (T, Hq + 2 * Hk, D), 1.2, dt)
        q, k, v = qkv.split([Hq, Hk, Hk], 1)
    else:
        q, k, v = (_normal(g, (T, H, D), 1.2, dt) for H in (Hq, Hk, Hk))
    s = dict(q=q, k=k, v=v, offsets=torch.tensor(_bounds(c), dtype=torch.int32, device="cuda"))
    if c["op"] == "attn_bwd":
        s["do"] = _normal(g, (T, Hq, D), 1e-2, dt)
        s["o"], s["lse"] = _attention(q, k, v, s["offsets"], c)
    return s


def _prepare_norm(c, g):
    dt, shape = DTYPES[c["dtype"]], (c["T"], c["C"])
    # a residual stream: an offset, and one value in a thousand thirty times larger
    x = torch.randn(shape, generator=g, device="cuda").add_(0.3)
    x = torch.where(torch.rand(shape, generator=g, device="cuda") < 1e-3, x * 30, x).to(dt)
    s = dict(x=x, w=None, b=None)
    if c["weight"]:
        s["w"] = (1 + _normal(g, (c["C"],), 0.2)).to(dt)
    if c["bias"]:
        s["b"] = _normal(g, (c["C"],), 0.2, dt)
    if c["op"] == "norm_bwd":
        s["dy"] = _normal(g, shape, 1e-2, dt)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = (_prepare_attn if case["op"].startswith("attn") else _prepare_norm)(case, g)
    s["case"] = case
    return s


# ----------------------------------------------------------------------------------------------- plain forms

def _by_group(x, Hk):
    """[n, heads, D] -> fp32 [Hk, heads / Hk * n, D]: the rows that share a key head."""
    n, H, D = x.shape
    return x.float().permute(1, 0, 2).reshape(Hk, H // Hk * n, D)


def _by_token(x, n):
    """Back to [n, heads, D]."""
    return x.reshape(-1, n, x.shape[-1]).permute(1, 0, 2)


def _pieces(c):
    """(begin, end) of runs of whole sequences whose scores are computed at once: short ones together, up to 2048
    tokens, and long ones alone, as most scores of several long ones would be masked."""
    pieces = []
    b = _bounds(c)
    for i, j in zip(b, b[1:]):
        if pieces and j - pieces[-1][0] <= 2048:
            pieces[-1] = pieces[-1][0], j
        elif i < j:
            pieces.append((i, j))
    return pieces


def _scores(q, k, i, j, offsets, c):
    """Scaled scores of the tokens i to j, [Hk, group * n, n], masked."""
    n = j - i
    at = torch.arange(i, j, device="cuda", dtype=torch.int32)
    of = torch.bucketize(at, offsets, right=True)
    hidden = of[:, None] != of[None, :]
    if c["causal"]:
        hidden |= at[:, None] < at[None, :]
    s = (q @ k.transpose(1, 2)).mul_(c["D"] ** -0.5)
    s.view(-1, n, n).masked_fill_(hidden, float("-inf"))
    return s


def _attention(q, k, v, offsets, c):
    Hq, Hk = c["Hq"], c["Hk"]
    o = torch.zeros((c["T"], Hq, c["D"]), dtype=q.dtype, device="cuda")
    lse = torch.full((Hq, c["T"]), float("-inf"), device="cuda")
    for i, j in _pieces(c):
        s = _scores(_by_group(q[i:j], Hk), _by_group(k[i:j], Hk), i, j, offsets, c)
        top = s.amax(-1, keepdim=True)
        p = s.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        o[i:j] = _by_token((p @ _by_group(v[i:j], Hk)).div_(total), j - i).to(q.dtype)
        lse[:, i:j] = (top + total.log()).view(Hq, j - i)
    return o, lse


def _attention_back(s, c):
    Hk, scale = c["Hk"], c["D"] ** -0.5
    dq, dk, dv = (torch.zeros(x.shape, dtype=x.dtype, device="cuda") for x in (s["q"], s["k"], s["v"]))
    for i, j in _pieces(c):
        n = j - i
        q, k, v, o, do = (_by_group(s[x][i:j], Hk) for x in ("q", "k", "v", "o", "do"))
        p = _scores(q, k, i, j, s["offsets"], c).sub_(s["lse"][:, i:j].reshape(Hk, -1, 1)).exp_()
        dv[i:j] = _by_token(p.transpose(1, 2) @ do, n).to(dv.dtype)
        ds = (do @ v.transpose(1, 2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
        dq[i:j] = _by_token(ds @ k, n).to(dq.dtype)
        dk[i:j] = _by_token(ds.transpose(1, 2) @ q, n).to(dk.dtype)
    return dq, dk, dv


def _unit(x, c):
    """(rows of mean 0 (where centred) and mean square 1, the factor that made them so), fp32."""
    x = x.float()
    if c["center"]:
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * r, r


def _plain(s):
    c = s["case"]
    if c["op"] == "attn_fwd":
        return list(_attention(s["q"], s["k"], s["v"], s["offsets"], c))
    if c["op"] == "attn_bwd":
        return list(_attention_back(s, c))
    x, w, b = s["x"], s["w"], s["b"]
    n, r = _unit(x, c)
    if c["op"] == "norm_fwd":
        y = n if w is None else n * w.float()
        return [(y if b is None else y + b.float()).to(x.dtype)]
    dy = s["dy"].float()
    dn = dy if w is None else dy * w.float()
    dx = dn - n * (dn * n).mean(-1, keepdim=True)
    if c["center"]:
        dx = dx - dn.mean(-1, keepdim=True)
    return [(dx * r).to(x.dtype), None if w is None else (dy * n).sum(0).to(w.dtype),
            None if b is None else dy.sum(0).to(b.dtype)]


def _framework(s):
    import all_gather_gb300 as tide
    c = s["case"]
    if c["op"] == "attn_fwd":
        return list(tide.attention(s["q"], s["k"], s["v"], s["offsets"], causal=c["causal"]))
    if c["op"] == "attn_bwd":
        return list(tide.attention_grad(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["offsets"],
                                        causal=c["causal"]))
    if c["op"] == "norm_fwd":
        return [tide.layer_norm(s["x"], s["w"], s["b"], eps=EPS, center=c["center"])]
    return list(tide.layer_norm_grad(s["dy"], s["x"], s["w"], s["b"], eps=EPS, center=c["center"]))


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------------ work, exact

def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    T = c["T"]
    if c["op"].startswith("attn"):
        b = _bounds(c)
        pairs = sum((j - i) * (j - i + 1) // 2 if c["causal"] else (j - i) ** 2 for i, j in zip(b, b[1:]))
        q, k, lse = T * c["Hq"] * c["D"] * e, T * c["Hk"] * c["D"] * e, T * c["Hq"] * 4
        if c["op"] == "attn_fwd":
            return {"bytes": 2 * q + 2 * k + lse, "flops": 4 * pairs * c["Hq"] * c["D"]}
        # the scores are not kept: five products
        return {"bytes": 4 * q + 4 * k + lse, "flops": 10 * pairs * c["Hq"] * c["D"]}
    n, small = T * c["C"], (c["weight"] + c["bias"]) * c["C"] * e
    if c["op"] == "norm_fwd":
        return {"bytes": 2 * e * n + small, "flops": 7 * n}
    return {"bytes": 3 * e * n + 2 * small, "flops": 14 * n}


def _exact_attn(s, c):
    """Each head of each sequence by itself, with a row's visible keys by comparison of positions."""
    back, scale, group = c["op"] == "attn_bwd", 1 / math.sqrt(c["D"]), c["Hq"] // c["Hk"]
    q, k, v = (s[x].double() for x in ("q", "k", "v"))
    o = torch.zeros_like(q)
    lse = torch.full((c["Hq"], c["T"]), float("-inf"), dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    b = _bounds(c)
    for i, j in zip(b, b[1:]):
        for h in range(c["Hq"] if j > i else 0):
            kh, vh = k[i:j, h // group], v[i:j, h // group]
            at = torch.arange(j - i, device="cuda")
            z = torch.einsum("td,sd->ts", q[i:j, h], kh) * scale
            if c["causal"]:
                z = torch.where(at[:, None] >= at[None, :], z, float("-inf"))
            if not back:
                lse[h, i:j] = torch.logsumexp(z, 1)
                o[i:j, h] = torch.softmax(z, 1) @ vh
                continue
            p = torch.exp(z - s["lse"][h, i:j].double()[:, None])
            g = s["do"][i:j, h].double()
            dz = p * (g @ vh.t() - torch.einsum("td,td->t", g, s["o"][i:j, h].double())[:, None])
            dv[i:j, h // group] += p.t() @ g
            dk[i:j, h // group] += scale * (dz.t() @ q[i:j, h])
            dq[i:j, h] = scale * (dz @ kh)
    return [dq, dk, dv] if back else [o, lse]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"].startswith("attn"):
        return _exact_attn(s, c)
    x, C = s["x"].double(), c["C"]
    mean = x.sum(-1, keepdim=True) / C if c["center"] else torch.zeros_like(x[:, :1])
    std = torch.sqrt(((x - mean) ** 2).sum(-1, keepdim=True) / C + EPS)
    n = (x - mean) / std
    w = torch.ones(C, dtype=torch.float64, device="cuda") if s["w"] is None else s["w"].double()
    if c["op"] == "norm_fwd":
        return [n * w if s["b"] is None else n * w + s["b"].double()]
    dy = s["dy"].double()
    g = dy * w
    along = n * ((g * n).sum(-1, keepdim=True) / C)
    dx = (g - along - (g.sum(-1, keepdim=True) / C if c["center"] else 0)) / std
    return [dx, None if s["w"] is None else torch.einsum("tc,tc->c", dy, n),
            None if s["b"] is None else dy.sum(0)]
