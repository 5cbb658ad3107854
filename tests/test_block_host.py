"""Host checks of attention and layer norm, no GPU needed: the C entry points refuse bad arguments before they touch the
device, with the documented status, and the wrappers refuse tensors of the wrong kind."""
import types

import pytest
import torch

import test_ops_wrappers as ow
from test_ops_host import A, b, refused, tide  # noqa: F401  (fixtures)
from test_ops_wrappers import BF16, OnGpu, OnGpu1, flat, graphs, leaves, put, world  # noqa: F401  (fixtures)


# ------------------------------------------------------------------------------------------ the C calls

def attention(b, **kw):
    d = dict(tokens=4, q_heads=4, k_heads=2, head_dim=64, causal=1, scale=0.125, offset_bytes=4, sequences=2, offsets=A,
             debug=0)
    d.update(kw)
    return b.AttentionDesc(**d)


def heads(b, p=A, ts=256, hs=64):
    return b.Heads(p, ts, hs)


@pytest.mark.parametrize("kw, status, match", [
    (dict(tokens=-1), 1, "tokens"), (dict(tokens=1 << 31), 1, "tokens"), (dict(q_heads=0), 1, "q_heads"),
    (dict(k_heads=0), 1, "k_heads"), (dict(q_heads=3), 1, "q_heads"), (dict(q_heads=65536), 1, "q_heads"),
    (dict(tokens=(1 << 31) - 512, q_heads=16), 1, "tokens"), (dict(head_dim=0), 1, "head_dim"),
    (dict(head_dim=60), 1, "head_dim"), (dict(head_dim=136), 3, "head_dim"), (dict(scale=0.0), 1, "scale"),
    (dict(scale=-1.0), 1, "scale"), (dict(scale=float("nan")), 1, "scale"), (dict(scale=float("inf")), 1, "scale"),
    (dict(offset_bytes=2), 1, "offset_bytes"), (dict(sequences=-1), 1, "sequences"),
    (dict(sequences=(1 << 31) - 1), 1, "sequences"), (dict(offsets=A + 2), 2, "offsets"), (dict(debug=1), 1, "debug"),
])
def test_attention_descriptor_refusals(tide, b, kw, status, match):
    h, d = heads(b), attention(b, **kw)
    refused(tide, status, match, b.tide_attention, d, h, h, h, h, A)
    refused(tide, status, match, b.tide_attention_grad, d, h, h, h, h, h, A, h, h, h, A, 1 << 40)
    refused(tide, 1, match, b.tide_attention_grad_workspace, d)


def test_attention_tensor_refusals(tide, b):
    ok = heads(b)

    def forward(at, bad):
        a = [ok] * 4
        a[at] = bad
        return attention(b), *a, A

    def backward(at, bad):
        a = [ok] * 8
        a[at] = bad
        return attention(b), *a[:5], A, *a[5:], A, 1 << 40

    for f, names, call in ((b.tide_attention, ("q", "k", "v", "o"), forward),
                           (b.tide_attention_grad, ("do", "q", "k", "v", "o", "dq", "dk", "dv"), backward)):
        for at, name in enumerate(names):
            refused(tide, 1, f"{name} is NULL", f, *call(at, None))
            refused(tide, 1, f"{name} is NULL", f, *call(at, heads(b, None)))
            refused(tide, 2, f"rows of {name} are not on", f, *call(at, heads(b, A + 8)))
            refused(tide, 2, f"rows of {name} are not on", f, *call(at, heads(b, ts=260)))
            refused(tide, 2, f"rows of {name} are not on", f, *call(at, heads(b, hs=68)))
            for bad in (dict(ts=0), dict(hs=0), dict(ts=-256), dict(ts=1 << 39), dict(hs=1 << 39)):
                refused(tide, 1, f"{name} has bad strides", f, *call(at, heads(b, **bad)))
            if name in ("o", "dq", "dk", "dv") and not (name == "o" and len(names) == 8):
                refused(tide, 1, f"rows of {name} overlap", f, *call(at, heads(b, ts=64)))
                refused(tide, 1, f"rows of {name} overlap", f, *call(at, heads(b, hs=32)))
    refused(tide, 1, "lse is NULL", b.tide_attention, attention(b), ok, ok, ok, ok, 0)
    refused(tide, 2, "lse", b.tide_attention, attention(b), ok, ok, ok, ok, A + 2)
    g = b.tide_attention_grad
    need = b.tide_attention_grad_workspace(attention(b))
    refused(tide, 1, "workspace", g, attention(b), ok, ok, ok, ok, ok, A, ok, ok, ok, A, need - 1)
    refused(tide, 1, "workspace", g, attention(b), ok, ok, ok, ok, ok, A, ok, ok, ok, 0, need)
    refused(tide, 2, "workspace", g, attention(b), ok, ok, ok, ok, ok, A, ok, ok, ok, A + 16, need)


def test_attention_of_nothing(tide, b):
    """No tokens: valid, whatever the tensors are."""
    d = attention(b, tokens=0)
    b.tide_attention(d, None, None, None, None, 0)
    b.tide_attention_grad(d, None, None, None, None, None, 0, None, None, None, 0, 0)
    assert b.tide_attention_grad_workspace(d) >= 256


@pytest.mark.parametrize("T, Hq, Hk, D", [(1, 1, 1, 8), (1000, 32, 4, 128), (8192, 32, 8, 128), (1 << 20, 64, 8, 64)])
def test_attention_workspace(tide, b, T, Hq, Hk, D):
    """delta, and at most as much again as fits two blocks' sums for each SM or so."""
    n = b.tide_attention_grad_workspace(attention(b, tokens=T, q_heads=Hq, k_heads=Hk, head_dim=D))
    assert T * Hq * 4 <= n <= T * Hq * 4 + 1024 + 4 * T + 8 * T * Hq * D


def norm(b, **kw):
    d = dict(rows=4, cols=64, dtype=0, center=1, weight=A, bias=A, eps=1e-5)
    d.update(kw)
    return b.NormDesc(**d)


@pytest.mark.parametrize("kw, status, match", [
    (dict(rows=-1), 1, "rows"), (dict(rows=1 << 61), 1, "rows"), (dict(cols=0), 1, "cols"),
    (dict(cols=(1 << 24) + 1), 1, "cols"), (dict(dtype=2), 3, "dtype"), (dict(eps=-1.0), 1, "eps"),
    (dict(eps=float("nan")), 1, "eps"), (dict(weight=A + 1), 2, "weight"), (dict(bias=A + 1), 2, "bias")])
def test_norm_descriptor_refusals(tide, b, kw, status, match):
    refused(tide, status, match, b.tide_layer_norm, norm(b, **kw), A, 64, A, 64)
    refused(tide, status, match, b.tide_layer_norm_grad, norm(b, **kw), A, 64, A, 64, A, 64, A, A, A, 1 << 40)
    refused(tide, 1, match, b.tide_layer_norm_grad_workspace, norm(b, **kw))


def test_norm_tensor_refusals(tide, b):
    f, g = b.tide_layer_norm, b.tide_layer_norm_grad
    for name, at in (("x", 0), ("y", 2)):
        for bad, status, match in ((0, 1, f"{name} is NULL"), (A + 1, 2, name)):
            a = [A, 64, A, 64]
            a[at] = bad
            refused(tide, status, match, f, norm(b), *a)
    refused(tide, 1, "x has stride", f, norm(b), A, -64, A, 64)
    refused(tide, 1, "y has stride", f, norm(b), A, 0, A, 63)
    for name, at in (("dy", 0), ("x", 2), ("dx", 4)):
        for bad, status, match in ((0, 1, f"{name} is NULL"), (A + 1, 2, name)):
            a = [A, 64, A, 64, A, 64]
            a[at] = bad
            refused(tide, status, match, g, norm(b), *a, A, A, A, 1 << 40)
    refused(tide, 1, "dx has stride", g, norm(b), A, 64, A, 64, A, 63, A, A, A, 1 << 40)
    refused(tide, 1, "both or neither", g, norm(b), A, 64, A, 64, A, 64, 0, A, A, 1 << 40)
    refused(tide, 1, "both or neither", g, norm(b, bias=None), A, 64, A, 64, A, 64, A, A, A, 1 << 40)
    refused(tide, 2, "dweight", g, norm(b), A, 64, A, 64, A, 64, A + 1, A, A, 1 << 40)
    need = b.tide_layer_norm_grad_workspace(norm(b))
    refused(tide, 1, "workspace", g, norm(b), A, 64, A, 64, A, 64, A, A, A, need - 1)
    refused(tide, 1, "workspace", g, norm(b), A, 64, A, 64, A, 64, A, A, 0, need)
    refused(tide, 2, "workspace", g, norm(b), A, 64, A, 64, A, 64, A, A, A + 16, need)
    assert b.tide_layer_norm_grad_workspace(norm(b, weight=None, bias=None)) == 0
    b.tide_layer_norm(norm(b, rows=0), 0, 0, 0, 0)


# ------------------------------------------------------------------------------------------ the wrappers

def calls(ops, kind=OnGpu):
    """Every operator on tensors of `kind`: name -> function of further arguments."""
    bf = lambda *s: put(torch.zeros(s, dtype=BF16), kind)  # noqa: E731
    q, k, x, w = bf(4, 2, 64), bf(4, 1, 64), bf(4, 64), bf(64)
    lse, off = put(torch.zeros(2, 4), kind), put(torch.tensor([0, 4], dtype=torch.int32), kind)
    return {
        "attention": lambda **kw: ops.attention(q, k, k, off, **kw),
        "attention_grad": lambda **kw: ops.attention_grad(q, q, k, k, q, lse, off, **kw),
        "layer_norm": lambda **kw: ops.layer_norm(x, w, w, **kw),
        "layer_norm_grad": lambda **kw: ops.layer_norm_grad(x, x, w, w, **kw),
    }


NAMES = ("attention", "attention_grad", "layer_norm", "layer_norm_grad")


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("passed", [None, 5, 7, "object"])
def test_memory_belongs_to_the_stream_of_the_work(world, name, passed):
    stream = types.SimpleNamespace(cuda_stream=7) if passed == "object" else passed
    calls(world.ops)[name](stream=stream)
    want = 5 if passed in (None, 5) else 7
    assert world.allocated and set(world.allocated) == {want}
    assert [a[-1] for _, a in world.lib.calls] == [want] and world.current == 5


@pytest.mark.parametrize("name", NAMES)
def test_tensors_on_another_device_than_the_current_are_refused(world, name):
    with pytest.raises(ValueError, match="device 1, and device 0 is current"):
        calls(world.ops, OnGpu1)[name]()
    assert not world.allocated and not world.lib.calls


@pytest.mark.parametrize("name", ["attention_grad", "layer_norm_grad"])
def test_workspace_on_another_device_is_refused(world, name):
    with pytest.raises(ValueError, match="workspace"):
        calls(world.ops)[name](workspace=put(torch.zeros(1 << 12, dtype=torch.uint8), OnGpu1))
    calls(world.ops)[name](workspace=put(torch.zeros(1 << 12, dtype=torch.uint8)))
    assert len(world.lib.calls) == 1


def test_tensors_that_do_not_fit_are_refused(world):
    ops = world.ops
    bf = lambda *s: put(torch.zeros(s, dtype=BF16))  # noqa: E731
    q, k = bf(4, 2, 64), bf(4, 1, 64)
    f32 = put(torch.zeros(4, 2, 64))
    with pytest.raises(TypeError, match="bfloat16"):
        ops.attention(f32, f32, f32)
    for a in ((bf(4, 64), k, k), (q, bf(5, 1, 64), k), (q, k, bf(4, 2, 64)), (q, bf(4, 1, 32), bf(4, 1, 32)),
              (q, k, put(torch.zeros(4, 1, 64)))):
        with pytest.raises(ValueError):
            ops.attention(*a)
    for off in (torch.zeros(3), torch.zeros((2, 2), dtype=torch.int32), torch.zeros(0, dtype=torch.int32),
                torch.zeros(8, dtype=torch.int64)[::2]):
        with pytest.raises(ValueError, match="offsets"):
            ops.attention(q, k, k, put(off))
    with pytest.raises(ValueError, match="offsets"):
        ops.attention(q, k, k, put(torch.zeros(3, dtype=torch.int32), OnGpu1))
    lse = put(torch.zeros(2, 4))
    for bad in (put(torch.zeros(4, 2)), put(torch.zeros(2, 4).double()), put(torch.zeros(4, 2).t())):
        with pytest.raises(ValueError, match="lse"):
            ops.attention_grad(q, q, k, k, q, bad)
        with pytest.raises(ValueError, match="lse"):
            ops.attention(q, k, k, out=(q, bad))
    with pytest.raises(ValueError, match="do has shape"):
        ops.attention_grad(k, q, k, k, q, lse)
    with pytest.raises(ValueError, match="contiguous last"):
        ops.attention(put(torch.zeros((4, 2, 128), dtype=BF16)[..., ::2]), k, k)
    x, w = bf(4, 64), bf(64)
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        ops.layer_norm(put(torch.zeros(4, 64).half()))
    with pytest.raises(TypeError, match="weight is"):
        ops.layer_norm(x, put(torch.zeros(64)))
    with pytest.raises(ValueError, match="bias has shape"):
        ops.layer_norm(x, w, bf(63))
    with pytest.raises(ValueError, match="rows, cols"):
        ops.layer_norm(q)
    with pytest.raises(ValueError, match="weight must be contiguous"):
        ops.layer_norm(x, put(torch.zeros(128, dtype=BF16)[::2]))
    with pytest.raises(ValueError, match="dbias goes with"):
        ops.layer_norm_grad(x, x, w, None, out=(x, w, w))
    assert not world.lib.calls


def differentiable(ops):
    """Every operator on leaves: name -> (leaves, function of further arguments that gives its outputs)."""
    bf = lambda *s: torch.zeros(s, dtype=BF16)  # noqa: E731
    qkv = leaves(bf(4, 2, 64), bf(4, 1, 64), bf(4, 1, 64))
    xwb = leaves(bf(4, 64), bf(64), bf(64))
    return {"attention": (qkv, lambda **kw: ops.attention(*qkv, **kw)),
            "layer_norm": (xwb, lambda **kw: (ops.layer_norm(*xwb, **kw),))}


@pytest.mark.parametrize("name", ["attention", "layer_norm"])
@pytest.mark.parametrize("curved", [False, True])
def test_second_derivatives_are_refused(graphs, name, curved):
    xs, f = differentiable(graphs.ops)[name]

    def loss():
        y = f()[0].float()
        return (y * y if curved else y).sum()

    for x in xs:
        grads = torch.autograd.grad(loss(), xs, create_graph=True)
        assert all(g.requires_grad for g in grads)
        with pytest.raises(RuntimeError, match="no second derivatives"):
            torch.autograd.grad(loss() + sum(g.float().pow(2).sum() for g in grads), x)


@pytest.mark.parametrize("stream", [None, 7])
@pytest.mark.parametrize("name", ["attention", "layer_norm"])
def test_operators_do_not_drop_the_graph(graphs, name, stream):
    xs, f = differentiable(graphs.ops)[name]
    f(stream=stream)[0].float().sum().backward()
    assert all(x.grad is not None and not x.grad.requires_grad for x in xs)
    with torch.no_grad():
        out = f(stream=stream)
        assert not any(t.requires_grad for t in out)
        f(out=out if name == "attention" else out[0])
    with pytest.raises(RuntimeError, match="out is given"):
        f(out=out if name == "attention" else out[0])
    for x in xs:
        x.requires_grad_(False)
    for x in xs:
        x.requires_grad_()
        assert f()[0].requires_grad
        x.requires_grad_(False)
    assert not any(t.requires_grad for t in f(stream=stream))


def test_lse_of_attention_has_no_gradient(graphs):
    o, lse = differentiable(graphs.ops)["attention"][1]()
    with pytest.raises(RuntimeError, match="lse has no gradient"):
        (o.float().sum() + lse.sum()).backward()


@pytest.mark.parametrize("name", NAMES)
def test_written_outputs_are_known_to_autograd(graphs, name):
    f = calls(graphs.ops)[name]
    out = f()
    ts = [out] if torch.is_tensor(out) else list(out)
    before = [t._version for t in ts]
    f(out=out)
    assert [t._version for t in ts] == [v + 1 for v in before]


def test_packed_structures_are_those_of_the_header(b):
    """The bytes that the wrappers pack are the ctypes structures'."""
    p = b.PackedCalls
    at = attention(b, tokens=7, sequences=3, scale=0.5, debug=2)
    assert p.attention(7, 4, 2, 64, 1, 0.5, 4, 3, A, 2) == bytes(at)
    n = norm(b, rows=9, cols=33, dtype=1, center=0, weight=A, bias=A + 64, eps=0.25)
    assert p.norm(9, 33, 1, 0, A, A + 64, 0.25) == bytes(n)
