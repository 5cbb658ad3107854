"""Cross entropy of tokens that are predicted well: losses near 0, where lse and the target's logit nearly cancel."""
import pytest
import torch

import ops_reference as ref
from test_gpu_ops import BF16, F32, close, gen, randn, tide  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def confident(seed, T, V, H, top=30.0, rivals=False):
    """Hidden states along their target's row, with target logits up to `top`; rivals: and as much along another row."""
    g = gen(seed)
    w = randn(g, (V, H), BF16, H ** -0.5)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    a = torch.linspace(1, top, T, device="cuda")[:, None]
    x = a * w[y].float()
    if rivals:
        x += a * w[(y + 1) % V].float() * torch.rand((T, 1), generator=g, device="cuda")
    return x.to(BF16), w, y


def exact(x, w, y):
    """(loss, lse, 1 - p of the target, target's logit), 64 bits, the loss without a cancellation."""
    z = x.double() @ w.double().t()
    at = torch.arange(len(y), device="cuda")
    zt = z[at, y].clone()
    lse = torch.logsumexp(z, 1)
    z[at, y] = -float("inf")
    loss = torch.nn.functional.softplus(torch.logsumexp(z, 1) - zt, threshold=1e9)
    return loss, lse, -torch.expm1(-loss), zt


def logit_errors(x, w, y):
    """Largest |error| of the other logits (every sum of the tensor cores cut once) and of the target's (an fp32 chain
    of H / 32 + 16)."""
    terms = x.double().abs() @ w.double().abs().t()
    H = x.shape[1]
    return (H + 8) * 2 * ref.U32 * terms.amax(1), (H / 32 + 16) * ref.U32 * (x.double() * w[y].double()).abs().sum(1)


CASES = [(64, 4096, 64, 30, False), (64, 4096, 4096, 30, False), (300, 1000, 1024, 40, False), (1, 5000, 2048, 30, False),
         (200, 3000, 4096, 40, True), (7, 32768, 2048, 25, True), (2100, 700, 256, 30, False), (40, 1, 64, 30, False),
         (40, 2, 64, 60, True)]


@pytest.mark.parametrize("T, V, H, top, rivals", CASES)
def test_losses_of_well_predicted_tokens(tide, T, V, H, top, rivals):
    """The loss's error is that of the logits, (1 - p) of it as d loss = sum of p_v (dz_v - dz_t) over the others, and
    roundings of its own; it is never negative."""
    x, w, y = confident(T + V + H, T, V, H, top, rivals)
    loss, lse = tide.linear_cross_entropy(x, w, y)
    assert (loss >= 0).all()
    want, wl, q, zt = exact(x, w, y)
    ev, et = logit_errors(x, w, y)
    own = 32 * ref.U32 * (1 + zt.abs() + wl.abs())  # the exponentials' arguments and results, the logarithm
    close(loss, want, 1.1 * q * (ev + et + own) + 8 * ref.U32 * want, "loss")
    close(lse, wl, et + q * ev + own, "lse")
    assert rivals or T == 1 or (want < 1e-4).any()


@pytest.mark.parametrize("T, V, H, top, rivals", [c for c in CASES if c[1] > 1])
def test_gradients_of_well_predicted_tokens(tide, T, V, H, top, rivals):
    """dz of a target is p - 1, however near 0, to the error of the target's logit: H / 32 roundings in each lane, each
    below U32 of the lane's share of the sum, taken as independent (six deviations), and the lanes' sum of 5 to 8."""
    x, w, y = confident(T + V + H + 1, T, V, H, top, rivals)
    _, wl, q, zt = exact(x, w, y)
    lse = wl.float()
    dloss = torch.rand(T, generator=gen(T), device="cuda") / T + 1e-3
    dx, dw = tide.linear_cross_entropy_grad(x, w, y, lse, dloss)
    ev, _ = logit_errors(x, w, y)
    x, w, s = x.double(), w.double(), dloss.double()[:, None]
    et = (6 * H ** 0.5 / 32 + 10) * ref.U32 * (x * w[y]).abs().sum(1) + 4 * ref.U32 * (zt - lse.double()).abs()
    at = torch.arange(T, device="cuda")
    d = torch.exp(x @ w.t() - lse.double()[:, None])
    err = d * (ev + 64 * ref.U32 * (1 + lse.double().abs()))[:, None]
    err[at, y] = d[at, y] * et
    d[at, y] = torch.expm1(zt - lse.double())
    d, err = d * s, (err + ref.U16 * d.abs()) * s
    n = max(T, V) + 64
    for got, want, e, terms, what in (
            (dx, d @ w, err @ w.abs(), d.abs() @ w.abs(), "dx"),
            (dw, d.t() @ x, err.t() @ x.abs(), d.abs().t() @ x.abs(), "dweight")):
        close(got, want, e + n * 2 * ref.U32 * terms + ref.U16 * want.abs() + 1e-30, what)


@pytest.mark.parametrize("T, V, H, pad", [(9, 300, 64, 0), (150, 1000, 72, 8), (70, 515, 63, 0), (513, 400, 256, 0),
                                          (33, 2000, 7, 1)])
def test_ignored_tokens_that_are_not_finite(tide, T, V, H, pad):
    """An ignored token's hidden state, lse and dloss give nothing, whatever they hold: the bits of a call in which they
    are zero."""
    g = gen(T)
    x, w = randn(g, (T, H + pad), BF16)[:, :H], randn(g, (V, H), BF16, H ** -0.5)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    off = torch.arange(T, device="cuda") % 4 == 1
    y[off] = -100
    d = torch.rand(T, generator=g, device="cuda")
    clean = torch.where(off[:, None], torch.zeros_like(x), x)
    loss, lse = tide.linear_cross_entropy(clean, w, y)
    want = tide.linear_cross_entropy_grad(clean, w, y, lse, d)
    assert (want[0][off] == 0).all()
    for value in (float("nan"), float("inf"), -float("inf"), 3e38):
        odd = torch.where(off[:, None], torch.full_like(x, value), x)
        got = tide.linear_cross_entropy(odd, w, y)[0]
        assert torch.equal(got, loss)
        fill = torch.full_like(d, value)
        got = tide.linear_cross_entropy_grad(odd, w, y, torch.where(off, fill, lse), torch.where(off, fill, d))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
