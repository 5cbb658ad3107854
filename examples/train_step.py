"""One transformer block trained on W virtual data-parallel ranks, all on one GPU.

    python examples/train_step.py --steps 20

A step is FSDP2's: the fp32 master shards are rounded to bf16 and placed as
full parameters (all-gather), every rank runs its own tokens forward and
backward, the ranks' bf16 gradients are folded into fp32 shards where they lie
(reduce-scatter), and each shard is updated.  Between the two collectives run
the operators that surround them in such a model: layer norms, norm of queries
and keys with the position rotation, attention, SwiGLU with 8-bit checkpoints,
and the vocabulary head with its cross entropy.  What is left, the
projections, is plain torch.
"""
from __future__ import annotations

import argparse
import os
import sys
from math import prod

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import all_gather_gb300 as tide  # noqa: E402
from all_gather_gb300 import autograd as ad  # noqa: E402

BF16 = torch.bfloat16


class Block:
    """Sizes and parameters of the model; grouped-query attention with a norm for each head."""

    def __init__(self, vocab=4099, hidden=256, heads=4, kv_heads=2, head_dim=64, ffn=704, context=128):
        self.vocab, self.hidden, self.heads, self.kv_heads = vocab, hidden, heads, kv_heads
        self.head_dim, self.ffn, self.context = head_dim, ffn, context
        h, d = hidden, head_dim
        self.shapes = {"embed": (vocab, h), "qkv": ((heads + 2 * kv_heads) * d, h), "q_norm": (d,), "k_norm": (d,),
                       "o": (h, heads * d), "gate_up": (2 * ffn, h), "down": (h, ffn), "head": (vocab, h)}
        self.table = tide.rope_table(context, d)
        self.positions = torch.arange(context, device="cuda")

    def init(self, name, g):
        shape = self.shapes[name]
        if len(shape) == 1:
            return torch.ones(shape, device="cuda")
        return torch.randn(shape, generator=g, device="cuda") * (0.5 if name == "embed" else shape[1] ** -0.5)

    def losses(self, p, tokens, targets):
        """Losses [context] of one sequence; p: the full parameters by name."""
        T, d, hq, hk = self.context, self.head_dim, self.heads, self.kv_heads
        norm = lambda x: ad.layer_norm(x, eps=1e-6, center=False)  # noqa: E731
        x = p["embed"][tokens]
        qkv = norm(x) @ p["qkv"].t()
        q, k, v = (t.view(T, -1, d) for t in qkv.split([hq * d, hk * d, hk * d], 1))
        q, k = ad.qk_norm_rope(q, k, self.table, self.positions, p["q_norm"], p["k_norm"])
        x = x + ad.attention(q, k, v).reshape(T, hq * d) @ p["o"].t()
        gate, up = (norm(x) @ p["gate_up"].t()).split(self.ffn, 1)
        x = x + ad.swiglu(gate, up) @ p["down"].t()
        return ad.linear_cross_entropy(norm(x), p["head"], targets)

    def plain_losses(self, p, tokens, targets):
        """The same in elementary operations, in the parameters' type."""
        T, d, hq, hk = self.context, self.head_dim, self.heads, self.kv_heads
        norm = lambda x: x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
        c, s = self.table.to(p["o"].dtype)[:, None].chunk(2, -1)

        def turned(x):
            a, b = x.chunk(2, -1)
            return torch.cat((a * c - b * s, b * c + a * s), -1)

        x = p["embed"][tokens]
        qkv = norm(x) @ p["qkv"].t()
        q, k, v = (t.view(T, -1, d) for t in qkv.split([hq * d, hk * d, hk * d], 1))
        q, k = turned(norm(q) * p["q_norm"]), turned(norm(k) * p["k_norm"])
        k, v = (t.repeat_interleave(hq // hk, 1) for t in (k, v))
        score = torch.einsum("thd,shd->hts", q, k) * d ** -0.5
        ahead = torch.ones(T, T, dtype=torch.bool, device="cuda").triu(1)
        attn = score.masked_fill(ahead, float("-inf")).softmax(-1)
        x = x + torch.einsum("hts,shd->thd", attn, v).reshape(T, hq * d) @ p["o"].t()
        gate, up = (norm(x) @ p["gate_up"].t()).split(self.ffn, 1)
        x = x + gate * gate.sigmoid() * up @ p["down"].t()
        return -(norm(x) @ p["head"].t()).log_softmax(-1).gather(1, targets[:, None])[:, 0]


def train(world=4, steps=20, lr=0.5, seed=0, model=None):
    """Mean loss of every step."""
    model = model or Block()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    names, shapes = list(model.shapes), list(model.shapes.values())
    # Gradients of every rank, one arena a rank: autograd adds into these views, the fold reads them in place.
    arenas = [torch.zeros(sum(-(-prod(s) // 128) * 128 for s in shapes), dtype=BF16, device="cuda")
              for _ in range(world)]
    grads, at = [[] for _ in range(world)], 0
    for s in shapes:
        for u in range(world):
            grads[u].append(arenas[u][at:at + prod(s)].view(s))
        at += -(-prod(s) // 128) * 128
    full = [torch.empty(s, dtype=BF16, device="cuda") for s in shapes]

    losses = []
    with tide.Plan(grads) as plan:
        S = plan.slot_numel
        master = torch.zeros(world, S, device="cuda")       # fp32 shards, rank-major
        shard_grads = torch.empty(world, S, device="cuda")
        for seg in plan.segments():  # scatter the initial parameters into the shards
            if seg["rank"] == 0:
                value = model.init(names[seg["param"]], g).reshape(-1)
            n, src, dst = seg["n_valid"], seg["src_elem"], seg["dst_elem"]
            master[seg["rank"], dst:dst + n] = value[src:src + n]
        bound = plan.bind_full(full)
        # Sequences to learn by heart: every rank has its own.
        text = torch.randint(0, model.vocab, (world, model.context + 1), generator=g, device="cuda")
        for _ in range(steps):
            plan.ag_place_f32(master, bound)
            total = torch.zeros((), device="cuda")
            for u in range(world):
                arenas[u].zero_()
                params = {}
                for name, p, view in zip(names, full, grads[u]):
                    params[name] = p.detach().requires_grad_()
                    params[name].grad = view
                loss = model.losses(params, text[u, :-1], text[u, 1:]).mean()
                loss.backward()
                total += loss.detach()
            plan.rs_fold(shard_grads, alpha=1.0 / world)
            master.add_(shard_grads, alpha=-lr)
            losses.append(total / world)
        out = [float(x) for x in losses]
        if tide.ops.device_status() != tide.TIDE_OK:
            raise RuntimeError("a device-side wait expired")
    return out


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--world", type=int, default=4)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=0.5)
    a = ap.parse_args()
    for i, x in enumerate(train(a.world, a.steps, a.lr)):
        print(f"step {i:3d}  loss {x:.4f}")
