"""The operators of the package itself on inputs that require a gradient: the same values, and the gradients of the
autograd functions."""
import pytest
import torch

from test_gpu_ops import BF16, F32, ce_inputs, gen, qk_inputs, randn, swiglu_inputs, tide  # noqa: F401  (fixture)

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
