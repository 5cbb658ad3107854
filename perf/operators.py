"""Cases, inputs and plain forms of the training-step operators, for measuring them.

Three operators, each in both directions:

* ``qk``     norm of queries and keys for each head, and the position rotation, in one pass
* ``ce``     vocabulary head and softmax cross entropy, without the logits in memory
* ``swiglu`` SwiGLU whose gate and up are kept in 8 bits for the backward pass

``own`` selects between the plain form (elementary torch operations in fp32, rounded once at the end) and the
framework's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
IGNORE = -100
BLOCK = 128      # columns that share one scale in an 8-bit checkpoint
FP8_MAX = 448.0  # largest e4m3 value
EPS = 1e-6


# ---------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one new token: what a generation step pays for the call itself
        dict(name="qk_fwd_one_token", op="qk_fwd", T=1, Hq=32, Hk=4, D=128, R=128, norm=True, interleaved=False,
             packed=True, dtype="bf16"),
        # a training micro-batch of a layer with 32 query and 4 key heads, read out of the packed projection
        dict(name="qk_fwd_32k", op="qk_fwd", T=32768, Hq=32, Hk=4, D=128, R=128, norm=True, interleaved=False,
             packed=True, dtype="bf16"),
        # an odd batch, fp32, interleaved pairs on part of a small head
        dict(name="qk_bwd_ragged_f32", op="qk_bwd", T=1003, Hq=7, Hk=3, D=96, R=48, norm=True, interleaved=True,
             packed=False, dtype="f32"),
        # the same training micro-batch on the way back
        dict(name="qk_bwd_32k", op="qk_bwd", T=32768, Hq=32, Hk=4, D=128, R=128, norm=True, interleaved=False,
             packed=True, dtype="bf16"),
        # a few tokens scored against a mid-size vocabulary: the weight's bytes count
        dict(name="ce_loss_few_tokens", op="ce_loss", T=7, V=32768, H=2048, dtype="bf16"),
        # a training micro-batch against a large vocabulary
        dict(name="ce_loss_8k", op="ce_loss", T=8192, V=131072, H=4096, dtype="bf16"),
        # a ragged last batch, odd vocabulary, with gradient
        dict(name="ce_grad_ragged", op="ce_grad", T=513, V=50001, H=2048, dtype="bf16"),
        # a training micro-batch with gradient
        dict(name="ce_grad_4k", op="ce_grad", T=4096, V=131072, H=4096, dtype="bf16"),
        # the tokens one expert of a mixture got
        dict(name="swiglu_fwd_expert", op="swiglu_fwd", T=67, F=768, packed=True, dtype="bf16"),
        # a dense layer's training micro-batch
        dict(name="swiglu_fwd_16k", op="swiglu_fwd", T=16384, F=14336, packed=True, dtype="bf16"),
        # odd rows and columns, fp32
        dict(name="swiglu_bwd_ragged_f32", op="swiglu_bwd", T=1001, F=1003, packed=False, dtype="f32"),
        # the dense layer on the way back
        dict(name="swiglu_bwd_16k", op="swiglu_bwd", T=16384, F=14336, packed=True, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: an odd multiple of 64, of 8 or of 1."""
    step = rng.choice((64, 64, 8, 1))
    return step * (((_log(rng, lo, hi) // step - 1) | 1))


def draw(rng):
    op = rng.choice(("qk_fwd", "qk_bwd", "ce_loss", "ce_grad", "swiglu_fwd", "swiglu_bwd"))
    if op.startswith("qk"):
        D = rng.choice((64, 80, 112, 128, 128, 128, 160, 256))
        Hk = rng.choice((1, 2, 4, 5, 8))
        Hq = Hk * rng.choice((1, 2, 4, 7, 8))
        R = rng.choice((D, D, D // 2))
        T = min(_log(rng, 1, 32768), 32768 * 36 * 128 // ((Hq + Hk) * D))
        dtype = rng.choice(("bf16", "bf16", "f32"))
        if dtype == "f32":
            T = max(1, T // 2)
        return dict(op=op, T=T, Hq=Hq, Hk=Hk, D=D, R=R, norm=rng.random() < 0.75, interleaved=rng.random() < 0.4,
                    packed=rng.random() < 0.5, dtype=dtype)
    if op.startswith("ce"):
        T, V, H = _log(rng, 1, 8192), _log(rng, 1000, 131072), _width(rng, 256, 4096)
        most = (8192 if op == "ce_loss" else 4096) * 131072 * 4096
        return dict(op=op, T=max(1, min(T, most // (V * H))), V=V, H=H, dtype="bf16")
    F = _width(rng, 256, 14336)
    T = min(_log(rng, 1, 32768), 16384 * 14336 // F)
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if dtype == "f32":
        T = max(1, T // 2)
    return dict(op=op, T=T, F=F, packed=rng.random() < 0.5, dtype=dtype)


# --------------------------------------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, scale=1.0, dtype=torch.float32):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return x.mul_(scale).to(dtype)


def _activations(g, shape, dtype):
    """N(0, 1) with one value in a thousand thirty times larger, as activations of large models have."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    far = torch.rand(shape, generator=g, device="cuda") < 1e-3
    return torch.where(far, x * 30, x).to(dtype)


def _prepare_qk(c, g):
    dt, T, Hq, Hk, D, R = DTYPES[c["dtype"]], c["T"], c["Hq"], c["Hk"], c["D"], c["R"]
    if c["packed"]:  # views of the packed q, k, v projection's output
        qkv = _normal(g, (T, (Hq + 2 * Hk) * D), 1.5, dt)
        q, k = qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    else:
        q, k = _normal(g, (T, Hq, D), 1.5, dt), _normal(g, (T, Hk, D), 1.5, dt)
    s = dict(q=q, k=k, wq=None, wk=None)
    if c["norm"]:
        s["wq"], s["wk"] = ((1 + _normal(g, (D,), 0.2)).to(dt) for _ in range(2))
    most = max(T, 4096)
    angle = torch.arange(most, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
    s["table"] = torch.cat((angle.cos(), angle.sin()), 1).float()  # [positions, R]: cosines, then sines
    # documents of several lengths in one batch: positions start again at each
    starts = torch.rand(T, generator=g, device="cuda") < 1 / 1024
    at = torch.arange(T, device="cuda")
    first = torch.where(starts, at, torch.zeros_like(at)).cummax(0).values
    s["positions"] = at - first + (int(torch.randint(0, most, (1,), generator=g, device="cuda")) if T == 1 else 0)
    if c["op"] == "qk_bwd":
        s["dq_out"], s["dk_out"] = _normal(g, (T, Hq, D), 1e-2, dt), _normal(g, (T, Hk, D), 1e-2, dt)
    return s


def _prepare_ce(c, g):
    dt, T, V, H = DTYPES[c["dtype"]], c["T"], c["V"], c["H"]
    w = _normal(g, (V, H), 1.0 / math.sqrt(H), dt)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    # normed hidden states that lean on their target's row: some tokens are predicted well, some not at all
    lean = 10 * torch.rand((T, 1), generator=g, device="cuda") ** 2
    x = (_normal(g, (T, H), 1.5) + lean * w[y].float()).to(dt)
    y = torch.where(torch.rand(T, generator=g, device="cuda") < 0.05, torch.full_like(y, IGNORE), y)  # padding
    if T == 1:
        y = y.clamp(min=0)
    s = dict(x=x, w=w, y=y)
    if c["op"] == "ce_grad":
        lse = torch.empty(T, device="cuda")
        for a in range(0, T, 1024):
            lse[a:a + 1024] = (x[a:a + 1024].float() @ w.float().t()).logsumexp(1)
        s["lse"] = lse
        s["dloss"] = torch.full((T,), 1.0 / max(1, int((y != IGNORE).sum())), device="cuda")
    return s


def _prepare_swiglu(c, g):
    dt, T, F = DTYPES[c["dtype"]], c["T"], c["F"]
    if c["packed"]:  # views of the packed gate and up projection's output
        both = _activations(g, (T, 2 * F), dt)
        gate, up = both[:, :F], both[:, F:]
    else:
        gate, up = _activations(g, (T, F), dt), _activations(g, (T, F), dt)
    if c["op"] == "swiglu_fwd":
        return dict(gate=gate, up=up)
    (g8, ge), (u8, ue) = _pack(gate.float()), _pack(up.float())
    return dict(ckpt=(g8, ge, u8, ue), dh=_normal(g, (T, F), 1e-2, dt))


def prepare(case, seed):
    g = _generator(seed)
    s = {"qk": _prepare_qk, "ce": _prepare_ce, "sw": _prepare_swiglu}[case["op"][:2]](case, g)
    s["case"] = case
    return s


# ----------------------------------------------------------------------------------------------- plain forms

def _rotated(x, table, positions, R, interleaved, back=False):
    """x [T, heads, D] fp32 with its first R columns rotated by the angles of its positions (back: by their negatives)."""
    cs = table[positions]
    c, s = cs[:, None, :R // 2], cs[:, None, R // 2:]
    if back:
        s = -s
    rot, rest = x[..., :R], x[..., R:]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = rot[..., :R // 2], rot[..., R // 2:]
        rot = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((rot, rest), -1)


def _qk_forward(x, w, s, c):
    f = x.float()
    if w is not None:
        f = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS) * w.float()
    return _rotated(f, s["table"], s["positions"], c["R"], c["interleaved"]).to(x.dtype)


def _qk_backward(d, x, w, s, c):
    dy = _rotated(d.float(), s["table"], s["positions"], c["R"], c["interleaved"], back=True)
    if w is None:
        return dy.to(x.dtype), None
    f = x.float()
    r = torch.rsqrt(f.square().mean(-1, keepdim=True) + EPS)
    n = f * r
    dw = (dy * n).sum((0, 1))
    dn = dy * w.float()
    return (r * (dn - n * (dn * n).mean(-1, keepdim=True))).to(x.dtype), dw.to(w.dtype)


def _pow2(e):
    """2^e as fp32 for whole e in [-126, 127], from its bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _pack(x):
    """(e4m3 values, biased exponents) of x [T, F] fp32: the smallest power of two that brings each block under 448."""
    T, F = x.shape
    B = -(-F // BLOCK)
    x = torch.nn.functional.pad(x, (0, B * BLOCK - F)).view(T, B, BLOCK)
    m, e = torch.frexp(x.abs().amax(-1))  # amax = m 2^e, 1/2 <= m < 1, and 448 = 7/8 2^9
    e = torch.where(m > 0, e - 9 + (m > 0.875), torch.zeros_like(e)).clamp(min=-126)
    q = (x * _pow2(-e)[..., None]).to(torch.float8_e4m3fn)
    return q.view(T, B * BLOCK)[:, :F].contiguous(), (e + 127).to(torch.uint8)


def _unpack(q, e):
    T, F = q.shape
    return q.float() * _pow2(e.int() - 127).repeat_interleave(BLOCK, 1)[:, :F]


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op == "qk_fwd":
        return [_qk_forward(s["q"], s["wq"], s, c), _qk_forward(s["k"], s["wk"], s, c)]
    if op == "qk_bwd":
        dq, dwq = _qk_backward(s["dq_out"], s["q"], s["wq"], s, c)
        dk, dwk = _qk_backward(s["dk_out"], s["k"], s["wk"], s, c)
        return [dq, dk, dwq, dwk]
    if op == "ce_loss":
        z = s["x"].float() @ s["w"].float().t()
        top = z.amax(1, keepdim=True)
        lse = (z - top).exp_().sum(1).log() + top[:, 0]
        kept = s["y"] != IGNORE
        zy = z.gather(1, s["y"].clamp(min=0)[:, None])[:, 0]
        return [torch.where(kept, lse - zy, torch.zeros_like(lse)), lse]
    if op == "ce_grad":
        x, w = s["x"].float(), s["w"].float()
        kept = s["y"] != IGNORE
        dz = (x @ w.t()).sub_(s["lse"][:, None]).exp_()
        dz.scatter_add_(1, s["y"].clamp(min=0)[:, None], torch.full_like(s["lse"], -1.0)[:, None])
        dz.mul_(torch.where(kept, s["dloss"], torch.zeros_like(s["dloss"]))[:, None])
        return [(dz @ w).to(s["x"].dtype), (dz.t() @ x).to(s["w"].dtype)]
    if op == "swiglu_fwd":
        g, u = s["gate"].float(), s["up"].float()
        (g8, ge), (u8, ue) = _pack(g), _pack(u)
        return [(g * torch.sigmoid(g) * u).to(s["gate"].dtype), g8, ge, u8, ue]
    g8, ge, u8, ue = s["ckpt"]
    g, u, dh = _unpack(g8, ge), _unpack(u8, ue), s["dh"].float()
    sg = torch.sigmoid(g)
    a = g * sg
    return [v.to(s["dh"].dtype) for v in (dh * u * (sg + a * (1 - sg)), dh * a, a * u)]


def _framework(s):
    import all_gather_gb300 as tide
    c = s["case"]
    op = c["op"]
    if op == "qk_fwd":
        return list(tide.qk_norm_rope(s["q"], s["k"], s["table"], s["positions"], s["wq"], s["wk"], eps=EPS,
                                      interleaved=c["interleaved"]))
    if op == "qk_bwd":
        return list(tide.qk_norm_rope_grad(s["dq_out"], s["dk_out"], s["q"], s["k"], s["table"], s["positions"],
                                           s["wq"], s["wk"], eps=EPS, interleaved=c["interleaved"]))
    if op == "ce_loss":
        return list(tide.linear_cross_entropy(s["x"], s["w"], s["y"], ignore_index=IGNORE))
    if op == "ce_grad":
        return list(tide.linear_cross_entropy_grad(s["x"], s["w"], s["y"], s["lse"], s["dloss"], ignore_index=IGNORE))
    if op == "swiglu_fwd":
        h, ckpt = tide.swiglu_ckpt8(s["gate"], s["up"])
        return [h, *ckpt]
    return list(tide.swiglu_ckpt8_grad(tide.Ckpt8(*s["ckpt"]), s["dh"]))


def run(state):
    return _framework(state) if own else _plain(state)


# ------------------------------------------------------------------------------------------------ work, exact

def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    op, T = c["op"], c["T"]
    if op.startswith("qk"):
        n = T * (c["Hq"] + c["Hk"]) * c["D"]
        small = T * 8 + min(T, 4096) * c["R"] * 4
        return {"bytes": (2 if op == "qk_fwd" else 3) * e * n + small, "flops": (10 if op == "qk_fwd" else 20) * n}
    if op == "ce_loss":
        return {"bytes": (T + c["V"]) * c["H"] * e + T * 16, "flops": 2 * T * c["V"] * c["H"]}
    if op == "ce_grad":  # the logits are not kept: one product more than the two gradients
        return {"bytes": 2 * (T + c["V"]) * c["H"] * e + T * 16, "flops": 6 * T * c["V"] * c["H"]}
    n, blocks = T * c["F"], 2 * T * -(-c["F"] // BLOCK)
    if op == "swiglu_fwd":
        return {"bytes": (3 * e + 2) * n + blocks, "flops": 10 * n}
    return {"bytes": (2 + 4 * e) * n + blocks, "flops": 14 * n}


def _exact_qk(s, c):
    out, grads = [], []
    h = c["R"] // 2
    cols = torch.arange(h, device="cuda")
    ia, ib = (2 * cols, 2 * cols + 1) if c["interleaved"] else (cols, cols + h)
    cs = s["table"].double()[s["positions"]][:, None, :]
    turn = torch.complex(cs[..., :h], cs[..., h:])
    for x, w, d in ((s["q"], s["wq"], s.get("dq_out")), (s["k"], s["wk"], s.get("dk_out"))):
        x = x.double()
        norm = torch.sqrt((x * x).sum(-1, keepdim=True) / c["D"] + EPS)
        unit = x / norm if w is not None else x
        if d is None:
            y = unit * w.double() if w is not None else unit.clone()
            z = torch.complex(y[..., ia], y[..., ib]) * turn
            y[..., ia], y[..., ib] = z.real, z.imag
            out.append(y)
            continue
        dy = d.double().clone()
        z = torch.complex(dy[..., ia], dy[..., ib]) * turn.conj()
        dy[..., ia], dy[..., ib] = z.real, z.imag
        if w is None:
            out.append(dy)
            grads.append(None)
            continue
        grads.append((dy * unit).sum((0, 1)))
        dy = dy * w.double()
        out.append((dy - unit * ((dy * unit).sum(-1, keepdim=True) / c["D"])) / norm)
    return out + grads


def exact(case, seed):
    c, s = case, prepare(case, seed)
    op = c["op"]
    if op.startswith("qk"):
        return _exact_qk(s, c)
    if op.startswith("ce"):
        if work(c)["flops"] > 1.4e13:  # over about 12 seconds in 64 bits
            return None
        x, w, y = s["x"].double(), s["w"].double(), s["y"]
        loss, lses, dx, dw = [], [], [], torch.zeros_like(w)
        for a in range(0, c["T"], 1024):
            xa, ya = x[a:a + 1024], y[a:a + 1024]
            z = xa @ w.t()
            kept, at = ya != IGNORE, torch.arange(len(ya), device="cuda")
            if op == "ce_loss":
                lse = torch.logsumexp(z, 1)
                lses.append(lse)
                loss.append(torch.where(kept, lse - z[at, ya.clamp(min=0)], 0.0))
                continue
            p = torch.exp(z - s["lse"][a:a + 1024].double()[:, None])
            p[at, ya.clamp(min=0)] -= 1.0
            p = p * torch.where(kept, s["dloss"][a:a + 1024].double(), 0.0)[:, None]
            dx.append(p @ w)
            dw += p.t() @ xa
        return [torch.cat(loss), torch.cat(lses)] if op == "ce_loss" else [torch.cat(dx), dw]
    if op == "swiglu_fwd":
        g, u = s["gate"].double(), s["up"].double()
        return [g / (1 + torch.exp(-g)) * u, None, None, None, None]
    g8, ge, u8, ue = s["ckpt"]
    scale = [torch.pow(2.0, e.double() - 127).repeat_interleave(BLOCK, 1)[:, :c["F"]] for e in (ge, ue)]
    g, u, dh = g8.double() * scale[0], u8.double() * scale[1], s["dh"].double()
    sg = 1 / (1 + torch.exp(-g))
    return [dh * u * sg * (1 + g * (1 - sg)), dh * g * sg, g * sg * u]
