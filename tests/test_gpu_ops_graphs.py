"""The operators of the package itself on inputs that require a gradient: the same values, and the gradients of the
autograd functions."""
import pytest
import torch

from test_gpu_ops import BF16, F32, ce_inputs, close, gen, qk_inputs, randn, swiglu_inputs, tide  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def inputs(name, dtype):
    """(leaves, the operator's call, the autograd functions' call)."""
    import all_gather_gb300 as tide
    from all_gather_gb300 import autograd as ad
    if name == "qk_norm_rope":
        q, k, wq, wk, table, pos = qk_inputs(1, 21, 4, 2, 64, 32, dtype, True, "plain")
        xs = [q, k, wq, wk]
        return xs, *(lambda f=f: torch.cat(f(q, k, table, pos, wq, wk, interleaved=True), 1)
                     for f in (tide.qk_norm_rope, ad.qk_norm_rope))
    if name == "linear_cross_entropy":
        x, w, y = ce_inputs(2, 40, 300, 72)
        return [x, w], lambda: tide.linear_cross_entropy(x, w, y)[0], lambda: ad.linear_cross_entropy(x, w, y)
    g, u = swiglu_inputs(3, 40, 300, dtype, "plain")
    return [g, u], lambda: tide.swiglu_ckpt8(g, u)[0], lambda: ad.swiglu(g, u)


@pytest.mark.parametrize("name, dtype", [("qk_norm_rope", BF16), ("qk_norm_rope", F32), ("linear_cross_entropy", BF16),
                                         ("swiglu_ckpt8", BF16), ("swiglu_ckpt8", F32)])
def test_outputs_lead_back_to_the_inputs(tide, name, dtype):
    xs, op, ad = inputs(name, dtype)
    plain = op()
    assert not plain.requires_grad
    d = randn(gen(4), plain.shape, plain.dtype)
    for x in xs:
        x.requires_grad_()
    got, want = op(), ad()
    assert torch.equal(got, plain) and torch.equal(want, plain)
    got = torch.autograd.grad(got, xs, d)
    want = torch.autograd.grad(want, xs, d)
    assert all(torch.equal(a, b) and a.abs().sum() > 0 for a, b in zip(got, want))


@pytest.mark.parametrize("name", ["qk_norm_rope", "linear_cross_entropy", "swiglu_ckpt8"])
def test_frozen_inputs(tide, name):
    """Each input alone has the gradient that it has among the others, and the frozen ones have none."""
    xs, op, _ = inputs(name, BF16)
    d = randn(gen(5), op().shape, op().dtype)
    for x in xs:
        x.requires_grad_()
    want = torch.autograd.grad(op(), xs, d)
    for i, x in enumerate(xs):
        for other in xs:
            other.requires_grad_(other is x)
        op().backward(d)
        assert torch.equal(x.grad, want[i]) and all(o.grad is None for o in xs if o is not x)
        x.grad = None


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("weights", [(True, False), (False, True), (False, False)])
def test_rotation_without_a_norm(tide, dtype, weights):
    """Queries or keys without a weight are rotated only, and their gradient is the reverse rotation."""
    import ops_reference as ref
    q, k, wq, wk, table, pos = qk_inputs(6, 33, 4, 2, 64, 32, dtype, True, "plain")
    wq, wk = (w if on else None for w, on in zip((wq, wk), weights))
    xs = [t.requires_grad_() for t in (q, k, wq, wk) if t is not None]
    out = tide.qk_norm_rope(q, k, table, pos, wq, wk, eps=1e-5)
    d = [randn(gen(7 + i), o.shape, dtype, 0.1) for i, o in enumerate(out)]
    torch.autograd.backward(out, d)
    M = ref.rotation(table, pos, 64, False)
    for x, w, g in ((q, wq, d[0]), (k, wk, d[1])):
        x, dx = x.detach(), x.grad
        want, dw, terms = ref.qk_backward(g, x, None if w is None else w.detach(), M, 1e-5)
        bound = ref.qk_backward_bound(g, x, None if w is None else w.detach(), M, want, dtype, 1e-5)
        close(dx, want, bound, "gradient")
        if w is not None:
            n = x.shape[0] * x.shape[1]
            close(w.grad, dw, ref.rounding(dtype) * dw.abs() + (n + 130) * 2 * ref.U32 * terms, "weight's gradient")
    assert all(x.grad is not None for x in xs)
