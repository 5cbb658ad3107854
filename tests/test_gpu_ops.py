"""The training-step operators on the GPU against plain 64-bit forms
(ops_reference), at the sizes, strides, types and values where they can go
wrong.  Every bound is the arithmetic's own (see ops_reference)."""
import math
import random

import pytest
import torch

import ops_reference as ref

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def tide():
    import all_gather_gb300
    all_gather_gb300.load_library()
    return all_gather_gb300


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def close(got, want, bound, what):
    got = got.double()
    bad = ~((got - want).abs() <= bound) & ~(torch.isnan(got) & torch.isnan(want)) & ~(got == want)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at "
                           f"{bad.nonzero()[0].tolist()}: {got[bad][0].item()} for {want[bad][0].item()} "
                           f"within {bound.expand_as(want)[bad][0].item()}")


class Framed:
    """A tensor of `shape` whose rows are `pad` elements apart inside a larger buffer of a known pattern, `shift`
    elements from its start; check() says whether anything outside the tensor changed."""

    def __init__(self, shape, dtype, pad=0, shift=0):
        inner = shape[-1] + pad
        n = inner * math.prod(shape[:-1])
        self.buf = torch.full((n + 2 * shift + 64,), 7.0, device="cuda", dtype=F32).to(dtype)
        strides = [1]
        for s in reversed((*shape[1:-1], inner) if len(shape) > 1 else ()):
            strides.insert(0, strides[0] * s)
        self.t = self.buf.as_strided(shape, strides, 32 + shift)
        self.idx = torch.ones_like(self.buf, dtype=torch.bool)
        self.idx.as_strided(shape, strides, 32 + shift).fill_(False)

    def check(self):
        assert (self.buf[self.idx].float() == 7.0).all(), "wrote outside the output"


# ------------------------------------------------------------------------------------------ rotary table

@pytest.mark.parametrize("scaling", [None, "linear", "by_parts"])
@pytest.mark.parametrize("n, R, base", [(1, 2, 10000.0), (517, 64, 10000.0), (131073, 128, 500000.0)])
def test_rope_table(tide, scaling, n, R, base):
    t = tide.rope_table(n, R, base=base, scaling=scaling, factor=8.0, low_freq_factor=1.0, high_freq_factor=4.0,
                        original=8192.0)
    f = ref.frequencies(R, base, scaling, 8.0, 1.0, 4.0, 8192.0).cuda()
    a = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * f
    # the angle's own rounding in 64 bits, and the fp32 store
    close(t, torch.cat((a.cos(), a.sin()), 1), torch.tensor(2.0 ** -24 + n * 2.0 ** -48, device="cuda"), "table")


# ------------------------------------------------------------------------------------------ head norm with rotation

def qk_inputs(seed, T, Hq, Hk, D, R, dtype, norm, layout, pos_dtype=torch.int64):
    g = gen(seed)
    if layout == "packed":
        qkv = randn(g, (T, (Hq + 2 * Hk) * D), dtype, 1.5)
        q, k = qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    elif layout == "heads_first":
        q, k = (randn(g, (H, T, D), dtype, 1.5).transpose(0, 1) for H in (Hq, Hk))
    elif layout == "odd":
        q, k = (randn(g, (T * H * (D + 3) + 1,), dtype, 1.5)[1:].view(T, H, D + 3)[..., :D] for H in (Hq, Hk))
    else:
        q, k = randn(g, (T, Hq, D), dtype, 1.5), randn(g, (T, Hk, D), dtype, 1.5)
    w = [(1 + randn(g, (D,), F32, 0.3)).to(dtype) if norm else None for _ in range(2)]
    table, pos = None, torch.zeros(T, dtype=torch.int64, device="cuda")
    if R:
        P = 300
        a = torch.rand((P, R // 2), generator=g, device="cuda") * 6.28
        table = torch.cat((a.cos(), a.sin()), 1)
        pos = torch.randint(0, P, (T,), generator=g, device="cuda").to(pos_dtype)
    return q, k, w[0], w[1], table, pos


QK_CASES = [
    # T, Hq, Hk, D, R, dtype, interleaved, norm, layout, position dtype
    (1, 32, 4, 128, 128, BF16, False, True, "packed", torch.int64),
    (5, 32, 8, 128, 128, BF16, False, True, "heads_first", torch.int32),
    (3, 32, 8, 128, 128, BF16, True, False, "plain", torch.int64),
    (257, 7, 3, 96, 48, F32, True, True, "plain", torch.int64),
    (67, 4, 1, 64, 64, BF16, False, True, "packed", torch.int32),
    (67, 1, 1, 80, 32, BF16, False, True, "packed", torch.int64),
    (33, 5, 2, 80, 80, F32, False, True, "plain", torch.int64),
    (19, 2, 2, 112, 16, BF16, True, True, "plain", torch.int64),
    (19, 3, 2, 160, 160, BF16, False, False, "packed", torch.int64),
    (19, 3, 0, 256, 128, BF16, False, True, "plain", torch.int64),
    (19, 0, 3, 256, 256, F32, True, True, "plain", torch.int64),
    (9, 2, 1, 512, 512, BF16, False, True, "plain", torch.int64),
    (9, 2, 1, 504, 0, F32, False, True, "plain", torch.int64),
    (9, 2, 1, 8, 0, BF16, False, True, "plain", torch.int64),
    (9, 2, 1, 24, 16, BF16, False, True, "plain", torch.int64),
    # shapes and rows that the vector path does not take
    (33, 5, 2, 100, 100, BF16, False, True, "packed", torch.int64),
    (33, 5, 2, 100, 50, F32, True, True, "plain", torch.int64),
    (33, 5, 2, 128, 128, BF16, False, True, "odd", torch.int64),
    (33, 5, 2, 128, 24, F32, True, True, "odd", torch.int32),
    (5, 2, 1, 1, 0, F32, False, True, "plain", torch.int64),
    (5, 2, 1, 2, 2, BF16, True, False, "plain", torch.int64),
    (5, 2, 1, 1000, 1000, BF16, False, True, "plain", torch.int64),
    (3, 2, 1, 4096, 512, F32, False, True, "plain", torch.int64),
    # many tokens: a warp takes all heads of one
    (4099, 6, 1, 64, 64, BF16, False, True, "packed", torch.int64),
    (4099, 3, 2, 64, 32, F32, True, True, "plain", torch.int64),
    (5001, 2, 1, 36, 12, BF16, False, True, "plain", torch.int64),
]


@pytest.mark.parametrize("T, Hq, Hk, D, R, dtype, il, norm, layout, pdt", QK_CASES)
def test_qk_norm_rope(tide, T, Hq, Hk, D, R, dtype, il, norm, layout, pdt):
    q, k, wq, wk, table, pos = qk_inputs(T + D, T, Hq, Hk, D, R, dtype, norm, layout, pdt)
    outs = [Framed((T, H, D), dtype, pad=8 if layout != "odd" else 1, shift=8 if layout != "odd" else 3)
            for H in (Hq, Hk)]
    tide.qk_norm_rope(q, k, table, pos, wq, wk, eps=1e-5, interleaved=il, out=[o.t for o in outs])
    own = tide.qk_norm_rope(q, k, table, pos, wq, wk, eps=1e-5, interleaved=il)
    M = ref.rotation(table, pos.long(), D, il) if D <= 512 or T <= 8 else None
    for x, w, o, o2, name in ((q, wq, outs[0], own[0], "q"), (k, wk, outs[1], own[1], "k")):
        o.check()
        assert torch.equal(o.t, o2), name
        if x.shape[1]:
            y = ref.qk_forward(x, w, M, 1e-5)
            close(o.t, y, ref.qk_forward_bound(x, w, y, dtype, 1e-5), name)


@pytest.mark.parametrize("T, Hq, Hk, D, R, dtype, il, norm, layout, pdt", QK_CASES)
def test_qk_norm_rope_grad(tide, T, Hq, Hk, D, R, dtype, il, norm, layout, pdt):
    q, k, wq, wk, table, pos = qk_inputs(T + D + 1, T, Hq, Hk, D, R, dtype, norm, layout, pdt)
    g = gen(T * D)
    dqo, dko = randn(g, (T, Hq, D), dtype, 0.1), randn(g, (T, Hk, D), dtype, 0.1)
    odd = layout == "odd"
    outs = [Framed((T, H, D), dtype, pad=1 if odd else 16, shift=3 if odd else 0) for H in (Hq, Hk)]
    dws = [Framed((D,), dtype, shift=1 if odd else 0) if norm else None for _ in range(2)]
    dwt = [None if d is None else d.t for d in dws]
    args = (dqo, dko, q, k, table, pos, wq, wk)
    n = 1 << 22
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    tide.qk_norm_rope_grad(*args, eps=1e-5, interleaved=il, out=[outs[0].t, outs[1].t, *dwt], workspace=ws)
    own = tide.qk_norm_rope_grad(*args, eps=1e-5, interleaved=il)
    M = ref.rotation(table, pos.long(), D, il)
    for i, (x, w, d, name) in enumerate(((q, wq, dqo, "q"), (k, wk, dko, "k"))):
        outs[i].check()
        assert torch.equal(outs[i].t, own[i]), name
        H = x.shape[1]
        dx, dw, terms = ref.qk_backward(d, x, w, M, 1e-5)
        if H:
            close(outs[i].t, dx, ref.qk_backward_bound(d, x, w, M, dx, dtype, 1e-5), "d" + name)
        if norm:
            dws[i].check()
            assert torch.equal(dwt[i], own[2 + i])
            # each term to a dozen roundings and its row's r, the sum in chains of at most T * H + 64
            close(dwt[i], dw, ref.rounding(dtype) * dw.abs() + (T * H + D / 32 + 128) * 2 * ref.U32 * terms,
                  f"d{name}_weight")


def test_qk_gradient_against_differences(tide):
    """The directional derivative of sum(out * r) along a random direction, in 64 bits, against the kernel's
    gradients (central differences: relative error about h^2 = 1e-10, and fp32 gradients)."""
    T, Hq, Hk, D, R, h = 11, 3, 2, 64, 32, 1e-5
    q, k, wq, wk, table, pos = qk_inputs(3, T, Hq, Hk, D, R, F32, True, "plain")
    g = gen(4)
    M = ref.rotation(table, pos, D, False)
    for x, w, i in ((q, wq, 0), (k, wk, 1)):
        r = [randn(g, t.shape, F32) for t in (q, k)]
        got = tide.qk_norm_rope_grad(*r, q, k, table, pos, wq, wk, eps=1e-5)
        vx, vw = randn(g, x.shape, F32).double(), randn(g, w.shape, F32).double()
        f = lambda e: (ref.qk_forward(x.double() + e * vx, w.double() + e * vw, M, 1e-5) * r[i].double()).sum()  # noqa
        diff = (f(h) - f(-h)) / (2 * h)
        along = (got[i].double() * vx).sum() + (got[2 + i].double() * vw).sum()
        size = (got[i].double() * vx).abs().sum() + (got[2 + i].double() * vw).abs().sum()
        assert abs(diff - along) <= 1e-5 * size


def test_qk_in_place_on_the_packed_projection(tide):
    T, Hq, Hk, D = 45, 8, 2, 128
    q, k, wq, wk, table, pos = qk_inputs(8, T, Hq, Hk, D, D, BF16, True, "packed")
    rest = q.as_strided((T, Hk * D), (q.stride(0), 1), q.storage_offset() + (Hq + Hk) * D).clone()
    want = tide.qk_norm_rope(q.clone(), k.clone(), table, pos, wq, wk)
    tide.qk_norm_rope(q, k, table, pos, wq, wk, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(rest, q.as_strided((T, Hk * D), (q.stride(0), 1), q.storage_offset() + (Hq + Hk) * D))


def test_qk_broadcast_input(tide):
    """Keys of one head read as four (stride 0), and their gradient per head."""
    q, k, wq, wk, table, pos = qk_inputs(9, 21, 4, 1, 64, 64, BF16, True, "plain")
    a = tide.qk_norm_rope(q, k.expand(21, 4, 64), table, pos, wq, wk)
    b = tide.qk_norm_rope(q, k.expand(21, 4, 64).contiguous(), table, pos, wq, wk)
    assert torch.equal(a[1], b[1])


@pytest.mark.parametrize("D", [64, 100])
def test_qk_odd_values(tide, D):
    """A row of zeroes stays 0 through the norm, NaN stays in its row, and a position outside the table gives NaN in
    the rotated columns only."""
    q, k, wq, wk, table, pos = qk_inputs(10, 6, 2, 1, D, D // 2 // 2 * 2 if D == 100 else 32, BF16, True, "plain")
    R = table.shape[1]
    q[0, 0] = 0
    q[1, 1, 5] = float("nan")
    pos[3], pos[4] = -1, table.shape[0]
    o, _ = tide.qk_norm_rope(q, k, table, pos, wq, wk)
    assert (o[0, 0] == 0).all()
    assert torch.isnan(o[1, 1]).all() and not torch.isnan(o[1, 0]).any()
    for t in (3, 4):
        assert torch.isnan(o[t, :, :R]).all() and not torch.isnan(o[t, :, R:]).any()
    assert not torch.isnan(o[5]).any() and not torch.isnan(o[2]).any()


def test_qk_no_tokens(tide):
    q, k, wq, wk, table, pos = qk_inputs(11, 0, 4, 2, 64, 64, BF16, True, "plain")
    o = tide.qk_norm_rope(q, k, table, pos, wq, wk)
    assert o[0].shape == (0, 4, 64)
    dwq, dwk = torch.full_like(wq, 5), torch.full_like(wk, 5)
    tide.qk_norm_rope_grad(q, k, q, k, table, pos, wq, wk, out=(q.clone(), k.clone(), dwq, dwk))
    assert (dwq == 0).all() and (dwk == 0).all()


def test_qk_offsets_past_32_bits(tide):
    T, H, D = 600_001, 28, 128  # 2.15e9 elements
    q = torch.empty((T, H, D), dtype=BF16, device="cuda")
    g = gen(12)
    q[:8] = randn(g, (8, H, D), BF16)
    q[8:-8] = 1
    q[-8:] = randn(g, (8, H, D), BF16)
    k = q[:, :1].contiguous()
    w = (1 + randn(g, (D,), F32, 0.3)).to(BF16)
    table = tide.rope_table(T, D)
    pos = torch.arange(T, device="cuda")
    o, _ = tide.qk_norm_rope(q, k, table, pos, w, w)
    for sl in (slice(0, 8), slice(T - 8, T)):
        y = ref.qk_forward(q[sl], w, ref.rotation(table, pos[sl], D, False), 1e-6)
        close(o[sl], y, ref.qk_forward_bound(q[sl], w, y, BF16, 1e-6), "rows")


# ------------------------------------------------------------------------------------------ cross entropy

def ce_inputs(seed, T, V, H, layout="plain", tdt=torch.int64, scale=1.0):
    g = gen(seed)
    pad, shift = {"plain": (0, 0), "wide": (8, 0), "odd": (1, 1)}[layout]
    x = randn(g, (T * (H + pad) + shift,), BF16, 1.5 * scale)[shift:].view(T, H + pad)[:, :H]
    w = randn(g, (V * (H + pad) + shift,), BF16, 1 / math.sqrt(H))[shift:].view(V, H + pad)[:, :H]
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    y = torch.where(torch.rand(T, generator=g, device="cuda") < 0.2, torch.full_like(y, -100), y)
    return x, w, y.to(tdt)


CE_CASES = [
    # T, V, H, layout, target dtype
    (1, 1, 1, "plain", torch.int64),
    (1, 5, 8, "plain", torch.int64),
    (1, 1000, 64, "plain", torch.int32),
    (2, 257, 63, "plain", torch.int64),
    (7, 513, 100, "plain", torch.int64),
    (64, 256, 128, "plain", torch.int64),
    (65, 255, 72, "wide", torch.int64),
    (128, 512, 64, "plain", torch.int32),
    (129, 1025, 200, "odd", torch.int64),
    (130, 129, 8, "odd", torch.int64),
    (256, 300, 264, "plain", torch.int64),
    (300, 2049, 136, "wide", torch.int64),
    (513, 777, 320, "plain", torch.int64),
    (40, 20001, 96, "plain", torch.int64),   # several pieces of the vocabulary
    (1025, 9000, 64, "plain", torch.int64),
]


@pytest.mark.parametrize("T, V, H, layout, tdt", CE_CASES)
def test_cross_entropy(tide, T, V, H, layout, tdt):
    x, w, y = ce_inputs(T + V + H, T, V, H, layout, tdt)
    fl, fs = Framed((T,), F32, shift=1), Framed((T,), F32, shift=2)
    tide.linear_cross_entropy(x, w, y, out=(fl.t, fs.t))
    fl.check(), fs.check()
    loss, lse, bound = ref.ce_loss(x, w, y)
    close(fl.t, loss, bound, "loss")
    close(fs.t, lse, bound, "lse")
    assert (fl.t[y == -100] == 0).all()
    again = tide.linear_cross_entropy(x, w, y)
    assert torch.equal(again[0], fl.t) and torch.equal(again[1], fs.t)


@pytest.mark.parametrize("T, V, H, layout, tdt", CE_CASES)
def test_cross_entropy_grad(tide, T, V, H, layout, tdt):
    x, w, y = ce_inputs(T + V + H + 1, T, V, H, layout, tdt)
    g = gen(T)
    dloss = torch.rand(T, generator=g, device="cuda") / T
    lse = ref.ce_loss(x, w, y)[1].float()
    dloss[y == -100] = float("nan")  # does not count
    pad, shift = {"plain": (0, 0), "wide": (8, 8), "odd": (1, 1)}[layout]
    fx, fw = Framed((T, H), BF16, pad, shift), Framed((V, H), BF16, pad, shift)
    tide.linear_cross_entropy_grad(x, w, y, lse, dloss, out=(fx.t, fw.t))
    fx.check(), fw.check()
    dx, dw, bx, bw = ref.ce_grad(x, w, y, lse, dloss)
    close(fx.t, dx, bx, "dx")
    close(fw.t, dw, bw, "dweight")
    ax, aw = tide.linear_cross_entropy_grad(x, w, y, lse, dloss)
    assert torch.equal(ax, fx.t) and torch.equal(aw, fw.t)


def test_cross_entropy_gradient_against_differences(tide):
    """The mean loss along a random direction of x and w, in 64 bits, against the kernel's bf16 gradients."""
    T, V, H, h = 33, 400, 64, 1e-5
    x, w, y = ce_inputs(21, T, V, H)
    lse = tide.linear_cross_entropy(x, w, y)[1]
    n = int((y != -100).sum())
    dx, dw = tide.linear_cross_entropy_grad(x, w, y, lse, torch.full((T,), 1 / n, device="cuda"))
    g = gen(22)
    vx, vw = randn(g, x.shape, F32).double(), randn(g, w.shape, F32).double()
    f = lambda e: ref.ce_loss(x.double() + e * vx, w.double() + e * vw, y)[0].sum() / n  # noqa: E731
    diff = (f(h) - f(-h)) / (2 * h)
    a, b = dx.double() * vx, dw.double() * vw
    # dz and the gradients are each rounded to bf16: 2 * 2^-9 of the terms at most
    assert abs(diff - a.sum() - b.sum()) <= 2.0 ** -8 * (a.abs().sum() + b.abs().sum())


@pytest.mark.parametrize("shift", [0, 1, 3, 5])
@pytest.mark.parametrize("H", [1, 3, 9, 63, 101, 2047])
def test_cross_entropy_rows_on_any_boundary(tide, H, shift):
    """Rows that start on every 2-byte boundary, in and out: the same bits as from aligned rows."""
    T, V = 30, 270
    x, w, y = ce_inputs(H + shift, T, V, H)
    d = torch.full((T,), 0.01, device="cuda")
    pitch = -(-H // 8) * 8
    X, W = (torch.zeros((n, pitch), dtype=BF16, device="cuda") for n in (T, V))
    X[:, :H], W[:, :H] = x, w
    loss, lse = tide.linear_cross_entropy(X[:, :H], W[:, :H], y)
    want = tide.linear_cross_entropy_grad(X[:, :H], W[:, :H], y, lse, d)
    fx, fw = (torch.zeros(n * H + shift, dtype=BF16, device="cuda")[shift:].view(n, H) for n in (T, V))
    fx.copy_(x), fw.copy_(w)
    assert torch.equal(tide.linear_cross_entropy(fx, fw, y)[0], loss)
    ox, ow = Framed((T, H), BF16, 0, shift), Framed((V, H), BF16, 0, shift)
    tide.linear_cross_entropy_grad(fx, fw, y, lse, d, out=(ox.t, ow.t))
    ox.check(), ow.check()
    assert torch.equal(ox.t, want[0]) and torch.equal(ow.t, want[1])


@pytest.mark.parametrize("H, pad", [(100, 4), (1, 7), (65, 7), (130, 6), (63, 1)])
def test_cross_entropy_reads_and_writes_its_columns_only(tide, H, pad):
    """Rows on 16-byte boundaries whose length is not a multiple of 16 bytes: what lies between them is not read (it
    is NaN) and not written."""
    T, V = 150, 300
    x, w, y = ce_inputs(H, T, V, H)
    X, W = (torch.full((n, H + pad), float("nan"), dtype=BF16, device="cuda") for n in (T, V))
    X[:, :H], W[:, :H] = x, w
    a = tide.linear_cross_entropy(x, w, y)
    b = tide.linear_cross_entropy(X[:, :H], W[:, :H], y)
    assert torch.isfinite(b[0]).all() and torch.equal(a[0], b[0])
    d = torch.full((T,), 0.01, device="cuda")
    fx, fw = Framed((T, H), BF16, pad), Framed((V, H), BF16, pad)
    g = tide.linear_cross_entropy_grad(x, w, y, a[1], d)
    tide.linear_cross_entropy_grad(X[:, :H], W[:, :H], y, a[1], d, out=(fx.t, fw.t))
    fx.check(), fw.check()
    assert torch.equal(fx.t, g[0]) and torch.equal(fw.t, g[1])


@pytest.mark.parametrize("T", [3, 140])
def test_cross_entropy_targets_that_do_not_count(tide, T):
    x, w, y = ce_inputs(31, T, 600, 64)
    y[:] = -100
    loss, lse = tide.linear_cross_entropy(x, w, y)
    assert (loss == 0).all() and torch.isfinite(lse).all()
    dx, dw = tide.linear_cross_entropy_grad(x, w, y, lse, torch.ones(T, device="cuda"))
    assert (dx == 0).all() and (dw == 0).all()
    y[0], y[1], y[2] = 600, -1, 5
    loss, lse = tide.linear_cross_entropy(x, w, y)
    assert torch.isnan(loss[:2]).all() and torch.isfinite(loss[2:]).all()
    dx, dw = tide.linear_cross_entropy_grad(x, w, y, lse, torch.ones(T, device="cuda"))
    assert torch.isnan(dx[:2]).all() and torch.isfinite(dx[2:]).all()
    y7 = torch.where(y == -100, torch.full_like(y, 7), y)
    assert (tide.linear_cross_entropy(x, w, y7, ignore_index=7)[0][3:] == 0).all()


def test_cross_entropy_extreme_logits(tide):
    """Logits of +-1e4, rows with an infinite or NaN hidden state, and one that is all -inf."""
    T, V, H = 6, 700, 64
    x, w, y = ce_inputs(41, T, V, H)
    y = y.clamp(min=0)
    x[0] *= 1e4
    x[1], x[2] = float("inf"), float("nan")
    w[:, 0] = w[:, 0].abs() + 0.01
    x[3], x[4] = 0, 0
    x[3, 0], x[4, 0] = -3e38, 3e38
    w[:, 0] *= 4
    loss, lse = tide.linear_cross_entropy(x, w, y)
    want, wl, bound = ref.ce_loss(x[[0, 5]], w, y[[0, 5]])
    close(loss[[0, 5]], want, bound, "loss")
    assert torch.isnan(lse[2]) and not torch.isfinite(lse[1])
    z = (x[3:5].float() @ w.float().t())  # overflows in fp32 as the logits do
    want = torch.logsumexp(z, 1)
    both = torch.isfinite(want)
    assert torch.equal(torch.isfinite(lse[3:5]), both) and torch.equal(lse[3:5][~both], want[~both])


@pytest.mark.parametrize("T", [0, 1])
def test_cross_entropy_no_tokens(tide, T):
    x, w, y = ce_inputs(51, T, 100, 64)
    y[:] = -100
    loss, lse = tide.linear_cross_entropy(x, w, y)
    assert loss.shape == (T,)
    dw = torch.full_like(w, 3)
    tide.linear_cross_entropy_grad(x, w, y, lse, torch.ones(T, device="cuda"), out=(torch.empty_like(x), dw))
    assert (dw == 0).all()


def test_cross_entropy_workspace_contents_do_not_matter(tide):
    x, w, y = ce_inputs(61, 200, 9001, 72)
    a = tide.linear_cross_entropy(x, w, y)
    d = torch.full((200,), 0.01, device="cuda")
    b = tide.linear_cross_entropy_grad(x, w, y, a[1], d)
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    a2 = tide.linear_cross_entropy(x, w, y, workspace=ws)
    ws.fill_(255)
    b2 = tide.linear_cross_entropy_grad(x, w, y, a[1], d, workspace=ws)
    for p, q in zip((*a, *b), (*a2, *b2)):
        assert torch.equal(p, q)
    assert tide.ops.device_status() == tide.TIDE_OK


@pytest.mark.parametrize("grad", [False, True])
def test_cross_entropy_wait_that_runs_out(tide, grad):
    """A fill that never comes ends its product's waits after 50 ms each; the status says so once, and the next call
    is whole again."""
    from all_gather_gb300 import _binding as b
    x, w, y = ce_inputs(71, 300, 2000, 128)
    want = tide.linear_cross_entropy(x, w, y)
    assert tide.ops.device_status() == tide.TIDE_OK
    desc = tide.ops._ce_desc(x, w, y, -100)[0]
    desc.debug = tide.TIDE_DEBUG_SHORT_WAIT | tide.TIDE_DEBUG_SKIP_FILL
    stream = torch.cuda.current_stream().cuda_stream
    a, c = torch.empty_like(want[0]), torch.empty_like(want[0])
    if grad:
        n = b.tide_ce_grad_workspace(desc)
        ws, dx, dw = torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(x), torch.empty_like(w)
        b.tide_ce_grad(desc, want[1].data_ptr(), want[0].data_ptr(), dx.data_ptr(), 128, dw.data_ptr(), 128,
                       ws.data_ptr(), n, stream)
    else:
        n = b.tide_ce_loss_workspace(desc)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        b.tide_ce_loss(desc, a.data_ptr(), c.data_ptr(), ws.data_ptr(), n, stream)
    assert tide.ops.device_status() == tide.TIDE_ERR_TIMEOUT
    assert tide.ops.device_status() == tide.TIDE_OK
    again = tide.linear_cross_entropy(x, w, y)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


def test_cross_entropy_drawn_shapes(tide):
    r = random.Random(5)
    for i in range(25):
        T, V, H = (max(1, int(math.exp(r.uniform(0, math.log(n))))) for n in (700, 5000, 400))
        layout = r.choice(("plain", "wide", "odd"))
        x, w, y = ce_inputs(i, T, V, H, layout)
        loss, lse = tide.linear_cross_entropy(x, w, y)
        wl, ws, bound = ref.ce_loss(x, w, y)
        close(loss, wl, bound, f"loss {T, V, H, layout}")
        d = torch.rand(T, device="cuda", generator=gen(i))
        got = tide.linear_cross_entropy_grad(x, w, y, lse, d)
        dx, dw, bx, bw = ref.ce_grad(x, w, y, lse, d)
        close(got[0], dx, bx, f"dx {T, V, H, layout}")
        close(got[1], dw, bw, f"dweight {T, V, H, layout}")


# ------------------------------------------------------------------------------------------ SwiGLU with checkpoints

def swiglu_inputs(seed, rows, cols, dtype, layout):
    g = gen(seed)
    x = torch.randn((rows, 2 * cols + 3), generator=g, device="cuda")
    far = torch.rand(x.shape, generator=g, device="cuda") < 0.01
    x = torch.where(far, x * 100, x).to(dtype)
    if layout == "packed":
        x = x[:, :2 * cols].contiguous()
        return x[:, :cols], x[:, cols:]
    if layout == "odd":
        return x[:, 1:cols + 1], x[:, cols + 1:2 * cols + 1]
    return x[:, :cols].contiguous(), x[:, cols:2 * cols].contiguous()


SWIGLU_CASES = [(r, c, dt, lay) for dt in (BF16, F32) for r, c, lay in (
    (1, 1, "plain"), (1, 8, "plain"), (3, 127, "plain"), (2, 128, "packed"), (5, 129, "plain"), (4, 256, "packed"),
    (67, 768, "packed"), (9, 1000, "packed"), (9, 1003, "plain"), (7, 520, "odd"), (33, 2056, "plain"),
    (1025, 136, "packed"), (2, 14336, "packed"))]


@pytest.mark.parametrize("rows, cols, dtype, layout", SWIGLU_CASES)
def test_swiglu_ckpt8(tide, rows, cols, dtype, layout):
    gate, up = swiglu_inputs(rows + cols, rows, cols, dtype, layout)
    odd = layout == "odd"
    h = Framed((rows, cols), dtype, pad=3 if odd else 8, shift=1 if odd else 0)
    codes = [Framed((rows, cols), torch.float8_e4m3fn, shift=1 if odd else 0) for _ in range(2)]
    exps = [Framed((rows, -(-cols // 128)), torch.uint8, shift=3) for _ in range(2)]
    ckpt = tide.Ckpt8(codes[0].t, exps[0].t, codes[1].t, exps[1].t)
    tide.swiglu_ckpt8(gate, up, out=(h.t, ckpt))
    for f in (h, *codes, *exps):
        f.check()
    want = ref.swiglu(gate, up)
    close(h.t, want, ref.swiglu_bound(want, want, gate, dtype), "h")
    for x, q, e in ((gate, ckpt[0], ckpt[1]), (up, ckpt[2], ckpt[3])):
        wq, we = ref.encode(x)
        assert torch.equal(e.long(), we)
        assert torch.equal(q.double(), wq)
    own_h, own = tide.swiglu_ckpt8(gate, up)
    assert torch.equal(own_h, h.t) and all(torch.equal(a.view(torch.uint8), b.contiguous().view(torch.uint8))
                                           for a, b in zip(own, ckpt))


@pytest.mark.parametrize("need_h", [True, False])
@pytest.mark.parametrize("rows, cols, dtype, layout", SWIGLU_CASES)
def test_swiglu_ckpt8_grad(tide, rows, cols, dtype, layout, need_h):
    gate, up = swiglu_inputs(rows + cols + 1, rows, cols, dtype, layout)
    _, ckpt = tide.swiglu_ckpt8(gate, up)
    dh = randn(gen(rows), (rows, cols + 8), dtype, 0.1)[:, (1 if layout == "odd" else 0):][:, :cols]
    outs = [Framed((rows, cols), dtype, pad=3 if layout == "odd" else 8) for _ in range(3)]
    got = tide.swiglu_ckpt8_grad(ckpt, dh, out=[o.t for o in outs[:2]] + [outs[2].t if need_h else None])
    g, u = (q.double() * ref.pow2(e).repeat_interleave(128, 1)[:, :cols]
            for q, e in ((ckpt[0], ckpt[1]), (ckpt[2], ckpt[3])))
    want = ref.swiglu_grad(g, u, dh)
    terms = ((1 + g.abs()) * dh.double().abs() * u.abs(), want[1], want[2])
    for i in range(3):
        outs[i].check()
        if i < 2 or need_h:
            close(got[i], want[i], ref.swiglu_bound(want[i], terms[i], g, dtype), ("dgate", "dup", "h")[i])
    own = tide.swiglu_ckpt8_grad(ckpt, dh, need_h=need_h)
    assert torch.equal(own[0], got[0]) and torch.equal(own[1], got[1]) and (own[2] is None) == (not need_h)


def test_swiglu_gradient_against_differences(tide):
    rows, cols, h = 5, 200, 1e-5
    gate, up = swiglu_inputs(71, rows, cols, F32, "plain")
    _, ckpt = tide.swiglu_ckpt8(gate, up)
    g, u = (q.double() * ref.pow2(e).repeat_interleave(128, 1)[:, :cols]
            for q, e in ((ckpt[0], ckpt[1]), (ckpt[2], ckpt[3])))
    r = gen(72)
    dh, vg, vu = (randn(r, (rows, cols), F32) for _ in range(3))
    dg, du, _ = tide.swiglu_ckpt8_grad(ckpt, dh)
    f = lambda e: (ref.swiglu(g + e * vg.double(), u + e * vu.double()) * dh.double()).sum()  # noqa: E731
    diff = (f(h) - f(-h)) / (2 * h)
    a, b = dg.double() * vg, du.double() * vu
    assert abs(diff - a.sum() - b.sum()) <= 1e-5 * (a.abs().sum() + b.abs().sum())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_swiglu_odd_values(tide, dtype):
    """Zero blocks, infinities and NaN (they do not count for the scale), subnormals and the largest values."""
    gate = torch.zeros((8, 300), dtype=dtype, device="cuda")
    gate[1] = 1e-40
    gate[2, :5] = torch.tensor([float("inf"), -float("inf"), float("nan"), 3.0, -1e-3], dtype=dtype)
    gate[3] = 3.3e38
    gate[4, 7], gate[4, 130] = 448.0, 449.0
    gate[5] = -1000.0
    gate[6, ::3] = 1e30
    gate[6, 1::3] = 1e-30
    up = torch.ones_like(gate)
    h, ckpt = tide.swiglu_ckpt8(gate, up)
    wq, we = ref.encode(gate)
    assert torch.equal(ckpt.gate_exps.long(), we)
    q = ckpt.gate_codes.double()
    assert torch.equal(torch.isnan(q), torch.isnan(wq)) and torch.equal(q[~torch.isnan(q)], wq[~torch.isnan(q)])
    assert (h[0] == 0).all() and (h[5].float().abs() == 0).all()
    assert torch.isposinf(h[2, 0]) and torch.isnan(h[2, 2])
    assert torch.isfinite(tide.swiglu_ckpt8_grad(ckpt, up)[0][[0, 1, 4, 5]]).all()


def test_swiglu_empty(tide):
    for rows, cols in ((0, 64), (5, 0)):
        x = torch.zeros((rows, cols), dtype=BF16, device="cuda")
        h, ckpt = tide.swiglu_ckpt8(x, x)
        assert h.shape == (rows, cols) and ckpt.gate_exps.shape == (rows, -(-cols // 128))
        assert tide.swiglu_ckpt8_grad(ckpt, x)[0].shape == (rows, cols)


def test_swiglu_offsets_past_32_bits(tide):
    rows, cols = 150_001, 14336  # 2.15e9 elements
    gate = torch.zeros((rows, cols), dtype=BF16, device="cuda")
    g = gen(81)
    gate[-3:] = randn(g, (3, cols), BF16)
    up = gate.flip(1)
    h, ckpt = tide.swiglu_ckpt8(gate, up)
    want = ref.swiglu(gate[-3:], up[-3:])
    close(h[-3:], want, ref.swiglu_bound(want, want, gate[-3:], BF16), "h")
    assert torch.equal(ckpt.up_codes[-3:].double(), ref.encode(up[-3:])[0])
    dg, du, h2 = tide.swiglu_ckpt8_grad(ckpt, up, out=(gate, h, None))
    last = [t[-3:].contiguous() for t in ckpt]
    want = tide.swiglu_ckpt8_grad(tide.Ckpt8(*last), up[-3:].contiguous())
    assert torch.equal(dg[-3:], want[0]) and torch.equal(du[-3:], want[1])


# ------------------------------------------------------------------------------------------ streams and graphs

def all_ops(tide):
    """Calls of every operator on fixed inputs: name -> function(stream, workspace) -> outputs."""
    q, k, wq, wk, table, pos = qk_inputs(91, 50, 8, 2, 128, 128, BF16, True, "packed")
    x, w, y = ce_inputs(92, 150, 1000, 64)
    lse = tide.linear_cross_entropy(x, w, y)[1]
    d = torch.full((150,), 0.01, device="cuda")
    gate, up = swiglu_inputs(93, 40, 300, BF16, "packed")
    _, ckpt = tide.swiglu_ckpt8(gate, up)
    return {
        "rope_table": lambda s: [tide.rope_table(100, 64, stream=s)],
        "qk": lambda s: tide.qk_norm_rope(q, k, table, pos, wq, wk, stream=s),
        "qk_grad": lambda s: tide.qk_norm_rope_grad(q, k, q, k, table, pos, wq, wk, stream=s),
        "ce": lambda s: tide.linear_cross_entropy(x, w, y, stream=s),
        "ce_grad": lambda s: tide.linear_cross_entropy_grad(x, w, y, lse, d, stream=s),
        "swiglu": lambda s: (lambda r: [r[0], *[t.view(torch.uint8) for t in r[1]]])(
            tide.swiglu_ckpt8(gate, up, stream=s)),
        "swiglu_grad": lambda s: tide.swiglu_ckpt8_grad(ckpt, up.contiguous(), stream=s),
    }


def test_other_streams(tide):
    """On a side stream, current or passed, behind work that delays it: the same bits."""
    ops = all_ops(tide)
    want = {n: [t.clone() for t in f(None)] for n, f in ops.items()}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for n, f in ops.items():
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
            got = f(None)
            got2 = f(side.cuda_stream)
            got = [t.clone() for t in got] + [t.clone() for t in got2]
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[n] * 2)), n


def test_graph_capture(tide):
    ops = all_ops(tide)
    want = {n: [t.clone() for t in f(None)] for n, f in ops.items()}
    torch.cuda.synchronize()
    for n, f in ops.items():
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = f(None)
        for _ in range(2):
            for t in got:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want[n])), n


def test_launches_are_counted(tide):
    ops = all_ops(tide)
    for n, f in ops.items():
        before = tide.tide_launch_count()
        f(None)
        assert tide.tide_launch_count() > before, n
