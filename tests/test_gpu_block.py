"""Attention and layer norm as a program uses them: on streams, in graphs, under autograd, together with the other
operators of a transformer block, and with a device-side wait that runs out."""
import math

import pytest
import torch

import block_reference as ref
from test_gpu_attention import check_forward, heads, on_gpu
from test_gpu_ops import BF16, F32, gen, randn, tide  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def all_calls(tide):
    """Calls on fixed inputs that outlive them: name -> function of further arguments."""
    q, k, v = heads(gen(1), 700, 8, 2, 128, "packed")
    off = on_gpu([0, 300, 301, 690])
    o, lse = tide.attention(q, k, v, off)
    q6, k6, v6 = heads(gen(2), 500, 4, 4, 64, "plain")
    x, w = randn(gen(3), (300, 2048), BF16), randn(gen(4), (2048,), BF16)
    y = randn(gen(5), (70, 333), F32)
    wy = randn(gen(6), (333,), F32)
    return {
        "attention": lambda **kw: tide.attention(q, k, v, off, **kw),
        "attention_grad": lambda **kw: tide.attention_grad(q, q, k, v, o, lse, off, **kw),
        "attention_full": lambda **kw: tide.attention(q6, k6, v6, causal=False, **kw),
        "layer_norm": lambda **kw: [tide.layer_norm(x, w, w, **kw)],
        "layer_norm_grad": lambda **kw: list(tide.layer_norm_grad(x, x, w, w, **kw)),
        "layer_norm_grad_f32": lambda **kw: list(tide.layer_norm_grad(y, y, wy, wy, center=False, **kw)),
    }


@pytest.mark.parametrize("raw", [False, True])
def test_other_streams(tide, raw):
    """A passed stream behind work that delays it, while the current one fills all memory that it is handed."""
    ops = all_calls(tide)
    want = {n: [t.clone() for t in f()] for n, f in ops.items()}
    side = torch.cuda.Stream()
    here = torch.cuda.current_stream()
    for n, f in ops.items():
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(5_000_000)
        got = f(stream=side.cuda_stream if raw else side)
        assert torch.cuda.current_stream() == here
        filled = [torch.full((size,), 255, dtype=torch.uint8, device="cuda")
                  for size in (256, 4096, 65536, 400_000, 1 << 20, 3 << 20) for _ in range(8)]
        here.synchronize()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[n])), n
        del filled


def test_two_streams_at_once(tide):
    """The same calls side by side, again and again, give the same bits."""
    ops = all_calls(tide)
    want = {n: [t.clone() for t in f()] for n, f in ops.items()}
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [(n, f(stream=s)) for _ in range(5) for n, f in ops.items() for s in streams]
    torch.cuda.synchronize()
    for n, out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want[n])), n
    assert tide.device_status() == tide.TIDE_OK


def test_graph_capture(tide):
    ops = all_calls(tide)
    want = {n: [t.clone() for t in f()] for n, f in ops.items()}
    torch.cuda.synchronize()
    for n, f in ops.items():
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = f()
        for _ in range(2):
            for t in got:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want[n])), n


def test_two_graphs_share_a_workspace(tide):
    """A graph's replay starts from whatever the other one's left in the workspace, and reads the offsets that are there
    when it runs."""
    q, k, v = heads(gen(7), 300, 8, 1, 64, "plain")
    do = randn(gen(8), (300, 8, 64), BF16)
    off = on_gpu([0, 300])
    o, lse = tide.attention(q, k, v, off)
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
    want = [t.clone() for t in tide.attention_grad(do, q, k, v, o, lse, off)]
    graphs = []
    for seed in (1, 2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = tide.attention_grad(do, q, k, v, o, lse, off, workspace=ws)
        graphs.append((graph, got))
    for _ in range(3):
        for graph, got in graphs:
            ws.fill_(255)
            graph.replay()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    off.copy_(on_gpu([0, 120]))
    o2, lse2 = tide.attention(q, k, v, off)
    want = tide.attention_grad(do, q, k, v, o2, lse2, off)
    o.copy_(o2), lse.copy_(lse2)
    graphs[0][0].replay()
    assert all(torch.equal(a, b) for a, b in zip(graphs[0][1], want))


def test_launches_are_counted(tide):
    for n, f in all_calls(tide).items():
        before = tide.tide_launch_count()
        f()
        assert tide.tide_launch_count() > before, n


def rel(a, b):
    return ((a.double() - b.double()).norm() / b.double().norm()).item()


def test_attention_in_autograd(tide):
    """Of views of a packed projection; an expanded incoming gradient; only some inputs with a gradient."""
    T, Hq, Hk, D = 150, 6, 2, 64
    qkv = randn(gen(9), (T, Hq + 2 * Hk, D), BF16, 0.8)
    off = on_gpu([0, 70, 150])
    grads = []
    for own in (True, False):
        x = (qkv if own else qkv.double()).detach().clone().requires_grad_()
        q, k, v = x.split([Hq, Hk, Hk], 1)
        if own:
            o = tide.attention(q, k, v, off)[0]
        else:
            a = ref.Attention(q, k, v, [0, 70, 150])
            o = a.tokens(a.o)
        (o.sum() + o[3:5].sin().sum()).backward()
        grads.append(x.grad)
    # p, ds, o and the results are rounded to bf16, each at most 2^-8 of its term: they add up at random
    assert grads[0].dtype == BF16 and rel(*grads) < 4 * ref.U16
    q, k, v = (t.detach().clone().requires_grad_(i == 1) for i, t in enumerate(qkv.split([Hq, Hk, Hk], 1)))
    tide.attention(q, k, v, off)[0].sum().backward()
    assert q.grad is None and v.grad is None and k.grad.shape == k.shape


def test_layer_norm_in_autograd(tide):
    for center in (True, False):
        x, w, b = randn(gen(10), (40, 320), F32), randn(gen(11), (320,), F32), randn(gen(12), (320,), F32)
        own = [t.clone().requires_grad_() for t in (x, w, b)]
        want = [t.double().requires_grad_() for t in (x, w, b)]
        tide.layer_norm(*own, center=center).sin().sum().backward()
        n = want[0] - want[0].mean(1, keepdim=True) if center else want[0]
        n = n * torch.rsqrt((n ** 2).mean(1, keepdim=True) + 1e-5)
        (n * want[1] + want[2]).sin().sum().backward()
        for a, c in zip(own, want):
            assert rel(a.grad, c.grad) < 1e-5


def test_a_captured_backward_pass_beside_a_live_graph(tide):
    """Forward and backward pass of copies of the leaves captured while a graph of the leaves themselves is alive."""
    x = randn(gen(13), (64, 256), BF16).requires_grad_()
    w = randn(gen(14), (256,), BF16).requires_grad_()
    alive = tide.layer_norm(x, w)

    def step(x, w):
        q = tide.layer_norm(x, w).view(64, 4, 64)
        return torch.autograd.grad(tide.attention(q, q[:, :2], q[:, 2:])[0], (x, w), torch.ones_like(q))

    copies = [t.detach().clone().requires_grad_() for t in (x, w)]
    want = step(*copies)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*copies)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    alive.sum().backward()
    assert torch.isfinite(x.grad).all()


def test_a_transformer_block(tide):
    """Norm, rotation, attention over packed sequences, SwiGLU and loss in a row, forward and backward, against the same
    in 64 bits: bf16 steps of 2^-8 at a dozen places add up to a few of them."""
    T, H, hq, hk, d, ffn, vocab = 96, 256, 4, 2, 64, 352, 500
    g = gen(15)
    off = on_gpu([0, 40, 96])
    pos = torch.cat((torch.arange(40), torch.arange(56))).cuda()
    table = tide.rope_table(64, d)
    shapes = {"x": (T, H), "n1": (H,), "qkv": ((hq + 2 * hk) * d, H), "nq": (d,), "nk": (d,), "o": (H, hq * d),
              "n2": (H,), "gu": (2 * ffn, H), "down": (H, ffn), "n3": (H,), "head": (vocab, H)}
    params = {n: (1 + randn(g, s, F32, 0.1) if len(s) == 1 else randn(g, s, F32, 1 if n == "x" else s[1] ** -0.5)).to(BF16)
              for n, s in shapes.items()}
    y = torch.randint(0, vocab, (T,), generator=g, device="cuda")

    def rms(x, w):
        return x * torch.rsqrt((x ** 2).mean(-1, keepdim=True) + 1e-6) * w

    def turned(x):
        c, s = table[pos, None, :d // 2].double(), table[pos, None, d // 2:].double()
        a, b = x[..., :d // 2], x[..., d // 2:]
        return torch.cat((a * c - b * s, b * c + a * s), -1)

    def own(p):
        x = p["x"]
        qkv = tide.layer_norm(x, p["n1"], eps=1e-6, center=False) @ p["qkv"].t()
        q, k, v = (t.view(T, -1, d) for t in qkv.split([hq * d, hk * d, hk * d], 1))
        q, k = tide.qk_norm_rope(q, k, table, pos, p["nq"], p["nk"])
        x = x + tide.attention(q, k, v, off)[0].reshape(T, -1) @ p["o"].t()
        gate, up = (tide.layer_norm(x, p["n2"], eps=1e-6, center=False) @ p["gu"].t()).split(ffn, 1)
        x = x + tide.swiglu_ckpt8(gate, up)[0] @ p["down"].t()
        return tide.linear_cross_entropy(tide.layer_norm(x, p["n3"], eps=1e-6, center=False), p["head"], y)[0]

    def plain(p):
        x = p["x"]
        qkv = rms(x, p["n1"]) @ p["qkv"].t()
        q, k, v = (t.view(T, -1, d) for t in qkv.split([hq * d, hk * d, hk * d], 1))
        a = ref.Attention(turned(rms(q, p["nq"])), turned(rms(k, p["nk"])), v, [0, 40, 96])
        x = x + a.tokens(a.o).reshape(T, -1) @ p["o"].t()
        gate, up = (rms(x, p["n2"]) @ p["gu"].t()).split(ffn, 1)
        x = x + torch.nn.functional.silu(gate) * up @ p["down"].t()
        return torch.nn.functional.cross_entropy(rms(x, p["n3"]) @ p["head"].t(), y, reduction="none")

    a = {n: t.clone().requires_grad_() for n, t in params.items()}
    c = {n: t.double().requires_grad_() for n, t in params.items()}
    la, lc = own(a), plain(c)
    assert rel(la, lc) < 4 * ref.U16
    la.mean().backward()
    lc.mean().backward()
    for n in shapes:  # the codes of gate and up are 2^-4 off at most, which their gradients have as noise
        assert rel(a[n].grad, c[n].grad) < 2 ** -4, n


def test_training_step_example_gradients():
    """The example's block against the same block in 64 bits: its gradients."""
    import os
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sys.path.insert(0, os.path.join(root, "examples"))
    try:
        import train_step
    finally:
        sys.path.pop(0)
    model = train_step.Block(vocab=300, context=48)
    g = gen(16)
    params = {n: model.init(n, g).to(BF16).requires_grad_() for n in model.shapes}
    tokens, targets = torch.randint(0, 300, (2, 48), generator=g, device="cuda")
    model.losses(params, tokens, targets).mean().backward()
    wide = {n: p.detach().double().requires_grad_() for n, p in params.items()}
    model.plain_losses(wide, tokens, targets).mean().backward()
    for n in params:
        assert rel(params[n].grad, wide[n].grad) < 2 ** -4, n


@pytest.mark.parametrize("T, Hq, Hk, D, causal", [(300, 4, 2, 128, True), (5000, 8, 8, 64, True), (700, 8, 1, 128, False)])
def test_what_a_lost_wait_leaves(tide, T, Hq, Hk, D, causal):
    """A tile that never comes: what depends on it is NaN, the rest is right, the status says so, and the next call is
    as if nothing had happened.  Nothing hangs: a fill is left out and waits end after 50 ms."""
    from all_gather_gb300 import _binding as b
    q, k, v = heads(gen(17), T, Hq, Hk, D, "plain")
    o, lse = tide.attention(q, k, v, causal=causal)
    grads = tide.attention_grad(q, q, k, v, o, lse, causal=causal)
    assert tide.device_status() == tide.TIDE_OK
    desc = b.AttentionDesc(T, Hq, Hk, D, int(causal), D ** -0.5, 8, 0, None,
                           tide.TIDE_DEBUG_SHORT_WAIT | tide.TIDE_DEBUG_SKIP_FILL)

    def h(t):
        return b.Heads(t.data_ptr(), t.stride(0), t.stride(1))

    stream = torch.cuda.current_stream().cuda_stream
    got = [torch.full_like(t, 5) for t in (o, lse, *grads)]
    ws = torch.zeros(b.tide_attention_grad_workspace(desc), dtype=torch.uint8, device="cuda")
    for forward in (True, False):
        if forward:
            b.tide_attention(desc, h(q), h(k), h(v), h(got[0]), got[1].data_ptr(), stream)
        else:
            b.tide_attention_grad(desc, h(q), h(q), h(k), h(v), h(o), lse.data_ptr(), *[h(t) for t in got[2:]],
                                  ws.data_ptr(), ws.numel(), stream)
        assert tide.device_status() == tide.TIDE_ERR_TIMEOUT
        assert tide.device_status() == tide.TIDE_OK
    for a, c in zip(got, (o, lse, *grads)):
        lost = torch.isnan(a)
        assert lost.any() and torch.equal(a[~lost], c[~lost])
    again = (*tide.attention(q, k, v, causal=causal), *tide.attention_grad(q, q, k, v, o, lse, causal=causal))
    assert all(torch.equal(a, c) for a, c in zip(again, (o, lse, *grads)))
    assert tide.device_status() == tide.TIDE_OK
