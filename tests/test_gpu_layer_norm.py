"""Layer norm and its gradient on the GPU against plain 64-bit forms (block_reference), at the sizes, strides, types and
values where they can go wrong."""
import pytest
import torch

import block_reference as ref
from test_gpu_ops import BF16, F32, Framed, close, gen, randn, tide  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

# rows, cols, dtype, layout
CASES = [
    (1, 1, F32, "plain"), (1, 5120, BF16, "plain"), (3, 2, BF16, "plain"), (5, 8, F32, "plain"), (7, 64, BF16, "plain"),
    (33, 100, BF16, "plain"), (33, 104, BF16, "padded"), (9, 1001, F32, "plain"), (9, 1001, BF16, "odd"),
    (67, 256, BF16, "padded"), (67, 264, F32, "padded"), (19, 768, BF16, "plain"), (2049, 512, BF16, "plain"),
    (300, 1024, F32, "plain"), (301, 2048, BF16, "padded"), (40, 4096, BF16, "plain"), (41, 4100, BF16, "plain"),
    (23, 5120, F32, "plain"), (1003, 1001, F32, "plain"), (5, 16384, BF16, "plain"), (5, 16392, F32, "plain"),
    (4, 32768, BF16, "plain"), (3, 32767, F32, "odd"), (3, 32776, BF16, "plain"), (2, 100_003, F32, "plain"),
    (5001, 72, F32, "plain"), (700, 8192, BF16, "plain"),
]


def rows_of(g, rows, cols, dtype, layout, scale=1.0):
    pad, shift = {"plain": (0, 0), "padded": (16, 0), "odd": (3, 1)}[layout]
    x = randn(g, (rows * (cols + pad) + shift,), F32, scale)
    return x.to(dtype)[shift:].view(rows, cols + pad)[:, :cols]


def inputs(rows, cols, dtype, layout, affine):
    g = gen(rows + cols)
    x = (rows_of(g, rows, cols, F32, layout) + 0.3)
    x[:, :: 97] *= 30
    x = rows_of(g, rows, cols, dtype, layout).copy_(x)
    w = (1 + randn(g, (cols,), F32, 0.3)).to(dtype) if "w" in affine else None
    b = randn(g, (cols,), F32, 0.3).to(dtype) if "b" in affine else None
    return x, w, b, rows_of(g, rows, cols, dtype, layout, 0.1)


@pytest.mark.parametrize("affine, center", [("wb", True), ("w", False), ("", True), ("b", False)])
@pytest.mark.parametrize("rows, cols, dtype, layout", CASES)
def test_layer_norm(tide, rows, cols, dtype, layout, affine, center):
    x, w, b, dy = inputs(rows, cols, dtype, layout, affine)
    n = ref.Norm(x, w, b, 1e-5, center)
    odd = layout == "odd"
    y = Framed((rows, cols), dtype, pad=3 if odd else 8, shift=1 if odd else 0)
    tide.layer_norm(x, w, b, center=center, out=y.t)
    y.check()
    close(y.t, n.y, n.bound(), "y")
    dx = Framed((rows, cols), dtype, pad=3 if odd else 8, shift=1 if odd else 0)
    dw, db = (None if t is None else Framed((cols,), dtype) for t in (w, b))
    got = tide.layer_norm_grad(dy, x, w, b, center=center,
                               out=(dx.t, None if dw is None else dw.t, None if db is None else db.t))
    want, bounds = n.grads(dy)
    for f, wanted, e, name in zip((dx, dw, db), want, bounds, ("dx", "dw", "db")):
        if f is not None:
            f.check()
            close(f.t, wanted, e, name)
    own = tide.layer_norm(x, w, b, center=center), *tide.layer_norm_grad(dy, x, w, b, center=center)
    for a, c in zip(own, (y.t, *got)):  # rows on other boundaries take other paths, with sums in another order
        if a is None:
            assert c is None
        elif layout == "plain" and cols % 8 == 0:
            assert torch.equal(a, c)
    assert all(torch.equal(a, c) for a, c in zip(own, (tide.layer_norm(x, w, b, center=center),
                                                       *tide.layer_norm_grad(dy, x, w, b, center=center)))
               if a is not None)


@pytest.mark.parametrize("cols", [512, 1001, 5120, 40000])
def test_written_over_an_input(tide, cols):
    x, w, b, dy = inputs(700, cols, BF16, "plain", "wb")
    y, grads = tide.layer_norm(x, w, b), tide.layer_norm_grad(dy, x, w, b)
    for over in range(2):
        xx, dd = x.clone(), dy.clone()
        got = tide.layer_norm_grad(dd, xx, w, b, out=((xx, dd)[over], torch.empty_like(w), torch.empty_like(b)))
        assert all(torch.equal(a, c) for a, c in zip(got, grads))
    assert torch.equal(tide.layer_norm(x, w, b, out=x), y)


@pytest.mark.parametrize("center", [True, False])
def test_broadcast_rows(tide, center):
    """A row that is read again and again: strides of 0."""
    x, w, b, dy = inputs(1, 640, BF16, "plain", "wb")
    xs, ds = x.expand(50, 640), dy.expand(50, 640)
    y = tide.layer_norm(xs, w, b, center=center)
    assert torch.equal(y, tide.layer_norm(x, w, b, center=center).expand(50, 640))
    got = tide.layer_norm_grad(ds, xs, w, b, center=center)
    n = ref.Norm(xs, w, b, 1e-5, center)
    want, bounds = n.grads(ds)
    for a, c, e, name in zip(got, want, bounds, ("dx", "dw", "db")):
        close(a, c, e, name)


def test_odd_values(tide):
    """A row far from 0, equal values, zeroes, the largest and smallest values, NaN and infinity in one row only."""
    for cols in (300, 304, 33000):
        x = randn(gen(1), (8, cols), F32)
        x[1] += 1000
        x[2] = 3.0
        x[3] = 0.0
        x[4] *= 1e-30
        x[5] *= 1e15
        x[6, 5] = float("nan")
        x[7, 5] = float("inf")
        y = tide.layer_norm(x, eps=1e-5)
        n = ref.Norm(x[:6], None, None, 1e-5, True)
        close(y[:6], n.y, n.bound(), "y")
        assert torch.isnan(y[6]).all() and not torch.isfinite(y[7]).any()
        assert (y[2:4] == 0).all()
        dy = randn(gen(2), (8, cols), F32)
        dx = tide.layer_norm_grad(dy, x)[0]
        want, bounds = n.grads(dy[:6])
        close(dx[:6], want[0], bounds[0], "dx")
        w = torch.ones(cols, device="cuda")
        dw = tide.layer_norm_grad(dy[:6], x[:6], w)[1]
        close(dw, want[1], bounds[1], "dw")


def test_gradient_against_differences(tide):
    rows, cols, h = 4, 200, 1e-5
    x, w, b, dy = inputs(rows, cols, F32, "plain", "wb")
    for center in (True, False):
        got = tide.layer_norm_grad(dy, x, w, b, center=center)
        xs = [t.double() for t in (x, w, b)]
        for i in range(3):
            d = torch.randn(xs[i].shape, generator=gen(i), device="cuda", dtype=torch.float64)

            def f(e):
                a, c, s = (t + e * d if j == i else t for j, t in enumerate(xs))
                m = a.mean(1, keepdim=True) if center else 0
                r = torch.rsqrt(((a - m) ** 2).mean(1, keepdim=True) + 1e-5)
                return (((a - m) * r * c + s) * dy.double()).sum()
            want = (f(h) - f(-h)) / (2 * h)
            assert abs((got[i].double() * d).sum() - want) <= 1e-5 * (got[i].double() * d).abs().sum()


def test_empty(tide):
    x = torch.zeros((0, 64), dtype=BF16, device="cuda")
    w = torch.ones(64, dtype=BF16, device="cuda")
    assert tide.layer_norm(x, w).shape == (0, 64)
    dx, dw, db = tide.layer_norm_grad(x, x, w, w)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()


def test_elements_past_32_bits(tide):
    rows, cols = 420_001, 5120  # 2.15e9 elements
    x = torch.zeros((rows, cols), dtype=BF16, device="cuda")
    g = gen(8)
    x[-3:] = randn(g, (3, cols), BF16)
    w = (1 + randn(g, (cols,), F32, 0.3)).to(BF16)
    y = tide.layer_norm(x, w, w)
    assert torch.equal(y[-3:], tide.layer_norm(x[-3:].clone(), w, w))
    dx, dw, db = tide.layer_norm_grad(x, x, w, w, out=(y, torch.empty_like(w), torch.empty_like(w)))
    want, bounds = ref.Norm(x[-3:], w, w, 1e-5, True).grads(x[-3:])
    close(dx[-3:], want[0], bounds[0], "dx")
    close(dw, want[1], bounds[1], "dw")
    close(db, want[2], bounds[2], "db")
