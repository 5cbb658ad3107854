"""The operators as autograd functions against plain fp32 forms of the same
model pieces, and the training-step example that runs them between the
placement and the fold."""
import math
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16 = torch.bfloat16


def rel(a, b):
    return ((a.float() - b.float()).norm() / b.float().norm()).item()


def leaf(x):
    return x.detach().clone().requires_grad_()


def test_qk_norm_rope_in_autograd():
    import all_gather_gb300 as tide
    from all_gather_gb300 import autograd as ad
    g = torch.Generator(device="cuda").manual_seed(1)
    T, hq, hk, D = 37, 4, 2, 64
    qkv = torch.randn(T, (hq + 2 * hk) * D, generator=g, device="cuda").to(BF16)
    wq, wk = (1 + 0.2 * torch.randn(2, D, generator=g, device="cuda")).to(BF16)
    table, pos = tide.rope_table(T, D), torch.arange(T, device="cuda")

    def plain(x, w):
        f = x.float()
        f = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6) * w.float()
        c, s = table[:, None, :D // 2], table[:, None, D // 2:]
        a, b = f[..., :D // 2], f[..., D // 2:]
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    grads = []
    for own in (True, False):
        x, a, b = leaf(qkv), leaf(wq), leaf(wk)
        q, k = x[:, :hq * D].view(T, hq, D), x[:, hq * D:(hq + hk) * D].view(T, hk, D)
        q, k = ad.qk_norm_rope(q, k, table, pos, a, b) if own else (plain(q, a), plain(k, b))
        (q.float().tanh().sum() + k.float().sin().sum()).backward()
        grads.append((x.grad, a.grad, b.grad))
    for own, want in zip(*grads):
        assert own.dtype == BF16 and rel(own, want) < 0.02  # q, k and their gradients rounded to bf16 on the way


def test_cross_entropy_in_autograd():
    from all_gather_gb300 import autograd as ad
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(100, 64, generator=g, device="cuda").to(BF16)
    w = (torch.randn(1000, 64, generator=g, device="cuda") / 8).to(BF16)
    y = torch.randint(0, 1000, (100,), generator=g, device="cuda")
    y[::7] = -100
    a, b = leaf(x), leaf(w)
    own = ad.linear_cross_entropy(a, b, y).sum() / 85
    own.backward()
    c, d = leaf(x.float()), leaf(w.float())
    want = torch.nn.functional.cross_entropy(c @ d.t(), y, reduction="sum") / 85
    want.backward()
    assert math.isclose(own.item(), want.item(), rel_tol=1e-5)
    assert rel(a.grad, c.grad) < 0.01 and rel(b.grad, d.grad) < 0.01


def test_swiglu_in_autograd():
    """Gradients at the 8-bit values: within the codes' error (at most 2^-4 relative a value) of the exact ones."""
    from all_gather_gb300 import autograd as ad
    g = torch.Generator(device="cuda").manual_seed(3)
    gu = torch.randn(65, 2 * 300, generator=g, device="cuda").to(BF16)
    a, b = leaf(gu), leaf(gu.float())
    ga, ua = a.split(300, 1)
    h = ad.swiglu(ga, ua)
    h.sum().backward()  # an expanded gradient
    gb, ub = b.split(300, 1)
    want = torch.nn.functional.silu(gb) * ub
    want.sum().backward()
    assert rel(h, want) < 2 ** -8
    assert rel(a.grad, b.grad) < 2 ** -4


def test_training_step_example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_step
    finally:
        sys.path.pop(0)
    a = train_step.train(world=2, steps=12)
    assert a[0] > math.log(4099) - 0.5  # an untrained model knows nothing: no better than a uniform guess
    assert a[-1] < a[0] - 1.0 and all(math.isfinite(x) for x in a)
