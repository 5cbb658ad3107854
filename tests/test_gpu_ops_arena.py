"""Gradients written by `out` into the arenas that the fold reads, rank by rank, and folded where they lie."""
import pytest
import torch

from test_gpu_ops import BF16, ce_inputs, qk_inputs, randn, gen, tide  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V, H", [(300, 64), (257, 63)])  # rows on 16-byte boundaries, and not
def test_gradients_go_straight_into_the_fold(tide, V, H):
    world, T, D = 4, 50, 128
    at, shapes = [], [(V, H), (D,), (D,)]
    n = 0
    for s in shapes:  # parameters one after the other, on 256-byte boundaries
        at.append(n)
        n += -(-torch.Size(s).numel() // 128) * 128
    arenas = torch.full((world, n), float("nan"), dtype=BF16, device="cuda")
    grads = [[arenas[u, a:a + torch.Size(s).numel()].view(s) for a, s in zip(at, shapes)] for u in range(world)]
    apart = []
    for u in range(world):
        x, w, y = ce_inputs(u, T, V, H)
        loss, lse = tide.linear_cross_entropy(x, w, y)
        d = torch.full((T,), 1 / T, device="cuda")
        q, k, wq, wk, table, pos = qk_inputs(u, T, 4, 2, D, D, BF16, True, "packed")
        dq, dk = randn(gen(u), (T, 4, D), BF16), randn(gen(u), (T, 2, D), BF16)
        tide.linear_cross_entropy_grad(x, w, y, lse, d, out=(torch.empty_like(x), grads[u][0]))
        tide.qk_norm_rope_grad(dq, dk, q, k, table, pos, wq, wk,
                               out=(torch.empty_like(dq), torch.empty_like(dk), grads[u][1], grads[u][2]))
        apart.append([tide.linear_cross_entropy_grad(x, w, y, lse, d)[1],
                      *tide.qk_norm_rope_grad(dq, dk, q, k, table, pos, wq, wk)[2:]])
    with tide.Plan(grads) as plan:
        folded = torch.zeros(world, plan.slot_numel, device="cuda")
        plan.rs_fold(folded, alpha=1.0 / world)
        for seg in plan.segments():
            want = apart[0][seg["param"]].float().reshape(-1)
            for u in range(1, world):
                want = want + apart[u][seg["param"]].float().reshape(-1)
            want = want * (1.0 / world)
            size, src, dst = seg["n_valid"], seg["src_elem"], seg["dst_elem"]
            assert torch.equal(folded[seg["rank"], dst:dst + size], want[src:src + size])
