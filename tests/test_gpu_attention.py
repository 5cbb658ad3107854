"""Attention over packed sequences and its gradient on the GPU against plain 64-bit forms (block_reference), at the
lengths, heads, strides, masks and values where they can go wrong."""
import random

import pytest
import torch

import block_reference as ref
from test_gpu_ops import BF16, F32, Framed, close, gen, randn, tide  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def heads(g, T, Hq, Hk, D, layout, scale=1.2):
    """q, k, v as views of a packed projection, heads first, with padded rows, or plain."""
    if layout == "packed":
        qkv = randn(g, (T, Hq + 2 * Hk, D), BF16, scale)
        return qkv.split([Hq, Hk, Hk], 1)
    if layout == "heads_first":
        return [randn(g, (H, T, D), BF16, scale).transpose(0, 1) for H in (Hq, Hk, Hk)]
    if layout == "padded":
        return [randn(g, (T, H, D + 8), BF16, scale)[..., 8:] for H in (Hq, Hk, Hk)]
    return [randn(g, (T, H, D), BF16, scale) for H in (Hq, Hk, Hk)]


def on_gpu(offsets, dtype=torch.int32):
    return None if offsets is None else torch.tensor(offsets, dtype=dtype, device="cuda")


# T, Hq, Hk, D, offsets, causal, layout
CASES = [
    (1, 4, 2, 128, None, True, "plain"),
    (1, 1, 1, 8, None, False, "packed"),
    (2, 3, 1, 64, [0, 1, 2], True, "packed"),
    (17, 8, 2, 128, [0, 17], True, "heads_first"),
    (61, 32, 4, 128, None, True, "packed"),
    (127, 2, 1, 80, None, True, "padded"),
    (128, 2, 2, 128, None, True, "plain"),
    (128, 2, 2, 64, None, False, "plain"),
    (129, 2, 1, 96, None, True, "packed"),
    (129, 2, 1, 96, None, False, "packed"),
    (255, 4, 1, 112, [0, 100, 101, 101, 255], True, "packed"),
    (256, 2, 2, 128, [0, 128, 256], True, "plain"),
    (257, 7, 1, 128, [0, 30, 257], False, "heads_first"),
    (300, 5, 5, 24, [3, 3, 40, 290], True, "padded"),      # rows before the first and behind the last sequence
    (300, 5, 5, 72, [3, 3, 40, 290], False, "packed"),
    (384, 4, 4, 16, [0, 384, 384], True, "plain"),
    (513, 8, 1, 128, [0, 512, 513], True, "packed"),
    (640, 6, 3, 120, None, True, "plain"),
    (700, 4, 2, 40, list(range(0, 701, 7)), True, "packed"),  # a hundred sequences
    (700, 4, 2, 64, list(range(0, 701, 70)), False, "packed"),
    (1000, 2, 1, 128, None, True, "packed"),
    (1000, 2, 2, 64, None, False, "heads_first"),
    (1111, 3, 3, 128, [0, 900, 1111], False, "packed"),
    (1500, 2, 1, 88, [0, 1, 2, 1400], True, "packed"),
    (40, 2, 2, 64, [0], True, "plain"),                      # no sequence
    (40, 2, 2, 64, [20, 20], False, "plain"),
]


def check_forward(tide, q, k, v, offsets, causal, got, a=None):
    a = a or ref.Attention(q, k, v, offsets, causal)
    o, lse = got
    none = ~a.some
    assert (o[none] == 0).all() and torch.isneginf(lse[:, none]).all()
    close(lse[:, a.some], a.lse[:, a.some], a.lse_bound()[:, a.some], "lse")
    close(o[a.some], a.tokens(a.o)[a.some], a.o_bound()[a.some], "o")
    return a


@pytest.mark.parametrize("T, Hq, Hk, D, offsets, causal, layout", CASES)
def test_attention(tide, T, Hq, Hk, D, offsets, causal, layout):
    q, k, v = heads(gen(T + D), T, Hq, Hk, D, layout)
    fo = Framed((T, Hq, D), BF16, pad=8, shift=8)
    lse = torch.full((Hq, T), 5.0, device="cuda")
    off = on_gpu(offsets)
    tide.attention(q, k, v, off, causal, out=(fo.t, lse))
    fo.check()
    check_forward(tide, q, k, v, offsets, causal, (fo.t, lse))
    own = tide.attention(q, k, v, on_gpu(offsets, torch.int64), causal)
    assert torch.equal(own[0], fo.t) and torch.equal(own[1], lse)


@pytest.mark.parametrize("T, Hq, Hk, D, offsets, causal, layout", CASES)
def test_attention_grad(tide, T, Hq, Hk, D, offsets, causal, layout):
    g = gen(T + D + 1)
    q, k, v = heads(g, T, Hq, Hk, D, layout)
    do = heads(g, T, Hq, 1, D, layout, 0.1)[0]
    off = on_gpu(offsets)
    o, lse = tide.attention(q, k, v, off, causal)
    outs = [Framed((T, H, D), BF16, pad=8, shift=8) for H in (Hq, Hk, Hk)]
    got = tide.attention_grad(do, q, k, v, o, lse, off, causal, out=[f.t for f in outs])
    for f in outs:
        f.check()
    a = ref.Attention(q, k, v, offsets, causal)
    want, bounds = a.grads(do, o, torch.where(a.some, lse, 0.0))
    for x, w, e, name in zip(got, want, bounds, ("dq", "dk", "dv")):
        assert (x[~a.some] == 0).all()
        close(x, w, e, name)
    own = tide.attention_grad(do, q, k, v, o, lse, on_gpu(offsets, torch.int64), causal)
    assert all(torch.equal(x, y) for x, y in zip(own, got))


def test_gradient_against_differences(tide):
    """Of the 64-bit form, along random directions: what the operator returns is its gradient."""
    T, Hq, Hk, D, offsets = 90, 4, 2, 64, [0, 50, 90]
    g = gen(5)
    q, k, v = heads(g, T, Hq, Hk, D, "plain", 0.7)
    do = randn(g, (T, Hq, D), BF16)
    o, lse = tide.attention(q, k, v, on_gpu(offsets))
    got = tide.attention_grad(do, q, k, v, o, lse, on_gpu(offsets))
    xs = [x.double() for x in (q, k, v)]
    h = 1e-5
    for i in range(3):
        d = torch.randn(xs[i].shape, generator=g, device="cuda", dtype=torch.float64)

        def f(e):
            y = [x + e * d if j == i else x for j, x in enumerate(xs)]
            a = ref.Attention(*y, offsets)
            return (a.tokens(a.o) * do.double()).sum()
        want = (f(h) - f(-h)) / (2 * h)
        # each element is within a few bf16 roundings of its terms, which add up at random: 2^-6 of the norm is eight
        # standard deviations
        size = got[i].double().norm() * d.norm() / d.numel() ** 0.5
        assert abs((got[i].double() * d).sum() - want) <= 2 ** -6 * size


def test_scales_and_large_scores(tide):
    """Scores in the hundreds, where one key takes all, and a scale that makes them all alike."""
    T, D = 200, 64
    for seed, amp, scale in ((1, 8.0, 0.5), (2, 20.0, 0.02), (3, 1.0, 1e-4), (4, 0.01, 50.0)):
        q, k, v = heads(gen(seed), T, 2, 1, D, "packed", amp)
        o, lse = tide.attention(q, k, v, scale=scale)
        a = ref.Attention(q, k, v, scale=scale)
        close(lse, a.lse, a.lse_bound(), "lse")
        close(o, a.tokens(a.o), a.o_bound(), "o")
        do = randn(gen(9), (T, 2, D), BF16)
        got = tide.attention_grad(do, q, k, v, o, lse, scale=scale)
        want, bounds = a.grads(do, o, lse)
        for x, w, e, name in zip(got, want, bounds, ("dq", "dk", "dv")):
            close(x, w, e, name)


def test_rising_scores(tide):
    """Every key's score is above those before it, so the running maximum moves at every tile."""
    T, D = 700, 64
    k = torch.zeros(T, 1, D, device="cuda")
    k[:, 0, 0] = torch.arange(T, device="cuda") / 8
    q = torch.zeros(T, 1, D, device="cuda")
    q[:, 0, 0] = 8
    q, k, v = q.to(BF16), k.to(BF16), randn(gen(3), (T, 1, D), BF16)
    for causal in (True, False):
        for kk in (k, k.flip(0)):
            got = tide.attention(q, kk, v, causal=causal)
            check_forward(tide, q, kk, v, None, causal, got)


BAD = [float("nan"), float("inf"), -float("inf")]


@pytest.mark.parametrize("value", BAD)
@pytest.mark.parametrize("causal", [True, False])
def test_what_is_not_seen_does_not_count(tide, value, causal):
    """NaN and infinities in tokens of no sequence, of another sequence, and (causal) of later tokens."""
    T, Hq, Hk, D, offsets = 400, 4, 2, 128, [5, 150, 390]
    off = on_gpu(offsets)
    for bad in (2, 395, 389, 200, 60):
        q, k, v = heads(gen(bad), T, Hq, Hk, D, "plain")
        do = randn(gen(bad + 1), (T, Hq, D), BF16, 0.1)
        for x in (q, k, v, do):
            x[bad, :, 3:9] = value
        o, lse = tide.attention(q, k, v, off, causal)
        a = ref.Attention(q, k, v, offsets, causal)
        clean = a.some & ~(a.see[:, bad]) & (torch.arange(T, device="cuda") != bad)
        close(lse[:, clean], a.lse[:, clean], a.lse_bound()[:, clean], f"lse {bad}")
        close(o[clean], a.tokens(a.o)[clean], a.o_bound()[clean], f"o {bad}")
        assert (o[~a.some] == 0).all()
        seen = a.see[:, bad] & a.some
        assert not torch.isfinite(o[seen][..., 3:9].float()).any()
        if bad not in (2, 395):
            assert not torch.isfinite(o[bad].float()).any()
        got = tide.attention_grad(do, q, k, v, o, lse, off, causal)
        want, bounds = a.grads(do, o, torch.where(a.some, lse, 0.0))
        for x, w, e, name in zip(got, want, bounds, ("dq", "dk", "dv")):
            fine = torch.isfinite(w) & torch.isfinite(e)
            assert fine[~a.some].all() and (bad < 60 or fine.any())
            close(x[fine], w[fine], e[fine], f"{name} {bad}")
            assert not torch.isfinite(x[torch.isnan(w)].float()).any()


def test_random_batches(tide):
    rng = random.Random(7)
    for i in range(40):
        D = 8 * rng.randint(1, 16)
        Hk = rng.choice((1, 2, 3))
        Hq = Hk * rng.choice((1, 2, 5))
        T = rng.randint(1, 600)
        offsets = sorted(rng.randint(0, T) for _ in range(rng.randint(1, 9)))
        causal = rng.random() < 0.6
        g = gen(i)
        q, k, v = heads(g, T, Hq, Hk, D, rng.choice(("plain", "packed", "heads_first", "padded")))
        got = tide.attention(q, k, v, on_gpu(offsets), causal)
        a = check_forward(tide, q, k, v, offsets, causal, got)
        do = randn(g, (T, Hq, D), BF16)
        grads = tide.attention_grad(do, q, k, v, *got, on_gpu(offsets), causal)
        want, bounds = a.grads(do, got[0], torch.where(a.some, got[1], 0.0))
        for x, w, e, name in zip(grads, want, bounds, ("dq", "dk", "dv")):
            close(x, w, e, name)


def test_offsets_that_mean_nothing(tide):
    """Decreasing offsets and offsets outside the tokens: nothing outside the outputs is written, and sequences that
    are whole are right."""
    T, H, D = 300, 2, 64
    q, k, v = heads(gen(1), T, H, H, D, "plain")
    for offsets in ([0, 200, 100, 300], [-5, 100, 1 << 30], [300, 200, 0], [1 << 31, 5], [-(1 << 40), 1 << 40]):
        off = on_gpu(offsets, torch.int64)
        fo = Framed((T, H, D), BF16, pad=8)
        lse = torch.empty((H, T), device="cuda")
        tide.attention(q, k, v, off, out=(fo.t, lse))
        fo.check()
        outs = [Framed((T, H, D), BF16, pad=8) for _ in range(3)]
        tide.attention_grad(q, q, k, v, fo.t, lse, off, out=[f.t for f in outs])
        for f in outs:
            f.check()
    got = tide.attention(q, k, v, on_gpu([-5, 100, 1 << 30], torch.int64))
    check_forward(tide, q, k, v, [0, 100, 300], True, got)


def test_empty(tide):
    q = torch.zeros((0, 4, 64), dtype=BF16, device="cuda")
    o, lse = tide.attention(q, q, q)
    assert o.shape == (0, 4, 64) and lse.shape == (4, 0)
    assert all(t.shape == (0, 4, 64) for t in tide.attention_grad(q, q, q, q, o, lse))


def test_elements_past_32_bits(tide):
    T, H, D, n = 270_000, 64, 128, 64  # 2.2e9 elements in sequences of 64
    q = torch.zeros((T, H, D), dtype=BF16, device="cuda")
    g = gen(4)
    q[-200:] = randn(g, (200, H, D), BF16)
    k = torch.zeros((T, 1, D), dtype=BF16, device="cuda")
    k[-200:] = randn(g, (200, 1, D), BF16)
    off = torch.arange(0, T + 1, n, device="cuda", dtype=torch.int32)  # the last tokens belong to none
    o, lse = tide.attention(q, k, k, off)
    dq, dk, dv = tide.attention_grad(q, q, k, k, o, lse, off)
    b = int(off[-1])
    a = b - n
    tail = [t[a:].contiguous() for t in (q, k)]
    off2 = on_gpu([0, n])
    o2, lse2 = tide.attention(tail[0], tail[1], tail[1], off2)
    close(o[a:b], o2[:n].double(), ref.U16 * 2 * o2[:n].double().abs() + 1e-3, "o")
    close(lse[:, a:b], lse2[:, :n].double(), 1e-4 + 0 * lse2[:, :n].double(), "lse")
    assert (o[b:] == 0).all() and torch.isneginf(lse[:, b:]).all() and (dq[b:] == 0).all() and (dk[b:] == 0).all()
    want = tide.attention_grad(tail[0], tail[0], tail[1], tail[1], o2, lse2, off2)
    for x, w in zip((dq, dk, dv), want):
        w = w[:n].double()
        close(x[a:b], w, 2 ** -6 * w.abs().amax() + 0 * w, "gradient")
