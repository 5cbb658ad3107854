"""The torch wrappers' own work, on the CPU with stand-ins for the library and
the streams: where memory is allocated, what is refused, what autograd sees."""
import contextlib
import types

import pytest
import torch

BF16 = torch.bfloat16


class OnGpu(torch.Tensor):
    """A CPU tensor that says it lies on a CUDA device."""
    dev = 0

    def get_device(self):
        return self.dev

    @property
    def is_cuda(self):
        return True


class OnGpu1(OnGpu):
    dev = 1


def put(t, kind=OnGpu):
    return t.as_subclass(kind)


class Library:
    """Takes every call for a success; keeps the name and the arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*a):
            if "workspace" in name:
                return 256
            self.calls.append((name, a))
            return 0
        return call


@pytest.fixture
def world(monkeypatch):
    """Device 0 is current, with stream 5; allocations note the stream that was current."""
    from all_gather_gb300 import _binding as b, ops
    w = types.SimpleNamespace(current=5, allocated=[], lib=Library(), ops=ops)

    @contextlib.contextmanager
    def stream(s):
        before, w.current = w.current, s.cuda_stream
        yield
        w.current = before

    def noting(f):
        def alloc(*a, **kw):
            w.allocated.append(w.current)
            kw.pop("device", None)
            return f(*a, **kw).zero_().as_subclass(OnGpu)
        return alloc

    monkeypatch.setattr(ops, "_current_device", lambda: 0)
    monkeypatch.setattr(ops, "_raw_stream", lambda d: w.current)
    monkeypatch.setattr(ops, "_empty", noting(torch.empty))
    monkeypatch.setattr(ops, "_empty_like", noting(torch.empty_like))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw: types.SimpleNamespace(cuda_stream=raw))
    monkeypatch.setattr(b, "packed_calls", lambda: w.lib)
    for name in ("tide_ce_loss", "tide_ce_grad", "tide_ce_loss_workspace", "tide_ce_grad_workspace", "tide_rope_table"):
        monkeypatch.setattr(b, name, getattr(w.lib, name))
    return w


def calls(ops, kind=OnGpu):
    """Every operator on tensors of `kind`: name -> function of further arguments."""
    bf = lambda *s: put(torch.zeros(s, dtype=BF16), kind)  # noqa: E731
    q, k, wt = bf(4, 2, 64), bf(4, 1, 64), bf(64)
    table, pos = put(torch.zeros(10, 64), kind), put(torch.zeros(4, dtype=torch.int64), kind)
    x, w, y = bf(4, 64), bf(100, 64), put(torch.zeros(4, dtype=torch.int64), kind)
    per = put(torch.zeros(4), kind)
    ckpt = ops.Ckpt8(*(put(torch.zeros(s, dtype=t), kind) for s, t in (
        ((4, 64), torch.float8_e4m3fn), ((4, 1), torch.uint8)) * 2))
    return {
        "qk_norm_rope": lambda **kw: ops.qk_norm_rope(q, k, table, pos, wt, wt, **kw),
        "qk_norm_rope_grad": lambda **kw: ops.qk_norm_rope_grad(q, k, q, k, table, pos, wt, wt, **kw),
        "linear_cross_entropy": lambda **kw: ops.linear_cross_entropy(x, w, y, **kw),
        "linear_cross_entropy_grad": lambda **kw: ops.linear_cross_entropy_grad(x, w, y, per, per, **kw),
        "swiglu_ckpt8": lambda **kw: ops.swiglu_ckpt8(x, x, **kw),
        "swiglu_ckpt8_grad": lambda **kw: ops.swiglu_ckpt8_grad(ckpt, x, **kw),
    }


NAMES = ("qk_norm_rope", "qk_norm_rope_grad", "linear_cross_entropy", "linear_cross_entropy_grad", "swiglu_ckpt8",
         "swiglu_ckpt8_grad")


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("passed", [None, 5, 7, "object"])
def test_memory_belongs_to_the_stream_of_the_work(world, name, passed):
    """Outputs and scratch memory are allocated with the launch's stream current: memory that is given back while the
    work runs then goes to later work on that stream only."""
    stream = types.SimpleNamespace(cuda_stream=7) if passed == "object" else passed
    calls(world.ops)[name](stream=stream)
    want = 5 if passed in (None, 5) else 7
    assert world.allocated and set(world.allocated) == {want}
    assert [a[-1] for _, a in world.lib.calls] == [want]
    assert world.current == 5


@pytest.mark.parametrize("name", NAMES)
def test_tensors_on_another_device_than_the_current_are_refused(world, name):
    """A call launches on the current device: tensors of another one are refused before anything is allocated."""
    with pytest.raises(ValueError, match="device 1, and device 0 is current"):
        calls(world.ops, OnGpu1)[name]()
    assert not world.allocated and not world.lib.calls


def test_workspace_and_table_on_another_device_are_refused(world):
    far = put(torch.zeros(1 << 12, dtype=torch.uint8), OnGpu1)
    for name in ("qk_norm_rope_grad", "linear_cross_entropy", "linear_cross_entropy_grad"):
        with pytest.raises(ValueError, match="workspace"):
            calls(world.ops)[name](workspace=far)
        calls(world.ops)[name](workspace=put(torch.zeros(1 << 12, dtype=torch.uint8)))
    assert len(world.lib.calls) == 3
    with pytest.raises(ValueError, match="out is on CUDA device 1"):
        world.ops.rope_table(10, 64, out=put(torch.zeros(10, 64), OnGpu1))
    world.ops.rope_table(10, 64, out=put(torch.zeros(10, 64)))
    assert len(world.lib.calls) == 4


# ------------------------------------------------------------------------------------------ autograd

@pytest.fixture
def graphs(world, monkeypatch):
    """The same, with every tensor on device 0 (autograd makes plain ones)."""
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    return world


def leaves(*ts):
    return [t.detach().requires_grad_() for t in ts]


def differentiable(ad):
    """Every differentiable operator: name -> (leaves, function that gives its first output)."""
    bf = lambda *s: torch.zeros(s, dtype=BF16)  # noqa: E731
    qk = leaves(bf(4, 2, 64), bf(4, 1, 64), bf(64), bf(64))
    table, pos = torch.zeros(10, 64), torch.zeros(4, dtype=torch.int64)
    ce = leaves(bf(4, 64), bf(100, 64))
    gu = leaves(bf(4, 64), bf(4, 64))
    return {
        "qk_norm_rope": (qk, lambda: ad.qk_norm_rope(qk[0], qk[1], table, pos, qk[2], qk[3])[0]),
        "linear_cross_entropy": (ce, lambda: ad.linear_cross_entropy(*ce, pos)),
        "swiglu": (gu, lambda: ad.swiglu(*gu)),
    }


@pytest.mark.parametrize("name", ["qk_norm_rope", "linear_cross_entropy", "swiglu"])
@pytest.mark.parametrize("curved", [False, True])
def test_second_derivatives_are_refused(graphs, name, curved):
    """A gradient with a graph of its own does not come back as a constant, whether or not the gradient that it was made
    from was one: going through it again is an error, for all leaves and for each of them."""
    from all_gather_gb300 import autograd as ad
    xs, f = differentiable(ad)[name]

    def loss():
        y = f().float()
        return (y * y if curved else y).sum()

    grads = torch.autograd.grad(loss(), xs, create_graph=True)
    assert len(grads) == len(xs) and all(g.requires_grad for g in grads)
    for x in xs:
        grads = torch.autograd.grad(loss(), xs, create_graph=True)
        with pytest.raises(RuntimeError, match="no second derivatives"):
            torch.autograd.grad(loss() + sum(g.float().pow(2).sum() for g in grads), x)
    grads = torch.autograd.grad(loss(), xs, create_graph=True)
    with pytest.raises(RuntimeError, match="no second derivatives"):
        (loss() + sum(g.float().pow(2).sum() for g in grads)).backward()


@pytest.mark.parametrize("name", ["qk_norm_rope", "linear_cross_entropy", "swiglu"])
def test_first_derivatives_have_no_graph(graphs, name):
    from all_gather_gb300 import autograd as ad
    xs, f = differentiable(ad)[name]
    f().float().sum().backward()
    assert all(x.grad is not None and not x.grad.requires_grad for x in xs)
    grads = torch.autograd.grad(f().float().sum(), xs, create_graph=True)
    (f().float().sum() + sum(g.detach().float().sum() for g in grads)).backward()  # used as numbers


def top_level(ops):
    """Every operator on leaves: name -> (leaves, function of further arguments that gives the outputs)."""
    bf = lambda *s: torch.zeros(s, dtype=BF16)  # noqa: E731
    qk = leaves(bf(4, 2, 64), bf(4, 1, 64), bf(64), bf(64))
    table, pos = torch.zeros(10, 64), torch.zeros(4, dtype=torch.int64)
    ce = leaves(bf(4, 64), bf(100, 64))
    gu = leaves(bf(4, 64), bf(4, 64))
    return {
        "qk_norm_rope": (qk, lambda **kw: ops.qk_norm_rope(qk[0], qk[1], table, pos, qk[2], qk[3], **kw)),
        "linear_cross_entropy": (ce, lambda **kw: ops.linear_cross_entropy(*ce, pos, **kw)),
        "swiglu_ckpt8": (gu, lambda **kw: ops.swiglu_ckpt8(*gu, **kw)),
    }


def flat(out):
    return [t for o in out for t in (o if isinstance(o, tuple) else (o,))]


@pytest.mark.parametrize("stream", [None, 7])
@pytest.mark.parametrize("name", ["qk_norm_rope", "linear_cross_entropy", "swiglu_ckpt8"])
def test_operators_do_not_drop_the_graph(graphs, name, stream):
    """Outputs of inputs that require a gradient lead back to them, each of the inputs by itself too; without them, or
    without recording, outputs are plain."""
    xs, f = top_level(graphs.ops)[name]
    out = f(stream=stream)
    assert out[0].requires_grad
    out[0].float().sum().backward()
    assert all(x.grad is not None for x in xs)
    for x in xs:
        x.requires_grad_(False)
    assert not any(t.requires_grad for t in flat(f(stream=stream)))
    for x in xs:
        x.requires_grad_()
        assert f()[0].requires_grad or (name == "qk_norm_rope" and f()[1].requires_grad)
        x.requires_grad_(False)
    xs[0].requires_grad_()
    with torch.no_grad():
        assert not any(t.requires_grad for t in flat(f(stream=stream)))


@pytest.mark.parametrize("name", ["qk_norm_rope", "linear_cross_entropy", "swiglu_ckpt8"])
def test_out_is_refused_where_a_gradient_is_wanted(graphs, name):
    xs, f = top_level(graphs.ops)[name]
    with torch.no_grad():
        out = f()
        f(out=out)
    n = len(graphs.lib.calls)
    with pytest.raises(RuntimeError, match="out is given"):
        f(out=out)
    assert len(graphs.lib.calls) == n


def test_lse_and_table_have_no_gradient(graphs):
    """What has no gradient here is refused instead of left out."""
    xs, f = top_level(graphs.ops)["linear_cross_entropy"]
    loss, lse = f()
    with pytest.raises(RuntimeError, match="lse has no gradient"):
        (loss.sum() + lse.square().sum()).backward()
    ckpt = top_level(graphs.ops)["swiglu_ckpt8"][1]()[1]
    assert not any(t.requires_grad for t in ckpt)
    q = torch.zeros(4, 2, 64, dtype=BF16)
    table, pos = torch.zeros(10, 64, requires_grad=True), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="table has no gradient"):
        graphs.ops.qk_norm_rope(q, q, table, pos)
    with torch.no_grad():
        graphs.ops.qk_norm_rope(q, q, table, pos)


@pytest.mark.parametrize("name", NAMES)
def test_written_outputs_are_known_to_autograd(graphs, name):
    """A tensor that a call wrote through `out` counts as changed, so that a graph that kept it refuses to go on."""
    f = calls(graphs.ops)[name]
    out = f()
    before = [t._version for t in flat(out) if t is not None]
    f(out=out)
    assert [t._version for t in flat(out) if t is not None] == [v + 1 for v in before]
    with torch.inference_mode():
        f(out=f())


def test_rotation_in_place_of_a_kept_tensor_is_noticed(graphs):
    q, k = (torch.zeros(4, 2, 64, dtype=BF16) for _ in range(2))
    w = torch.ones(64, requires_grad=True)
    y = (q.float() * w).sum() + (q * q.detach().requires_grad_()).sum()  # keeps q
    graphs.ops.qk_norm_rope(q, k, out=(q, k))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


# ------------------------------------------------------------------------------------------ the C calls

def test_strides_that_no_tensor_map_takes_are_refused_at_once():
    """Such a call used to fail half way, with kernels already under way."""
    from all_gather_gb300 import _binding as b, build
    build.build()
    a, far = 0x7F0000000000, 1 << 39  # an address that is never read

    def desc(x_stride=64, weight_stride=64):
        return b.CeDesc(4, 100, 64, a, x_stride, a, weight_stride, a, 8, -100)

    def refused(match, f, *args):
        before = b.tide_launch_count()
        with pytest.raises(b.TideError, match=match) as e:
            f(*args)
        assert e.value.status == b.TIDE_ERR_INVALID_ARG and b.tide_launch_count() == before

    for d in (desc(x_stride=far), desc(weight_stride=far)):
        refused("x_stride", b.tide_ce_loss, d, a, a, a, 1 << 50)
        refused("x_stride", b.tide_ce_grad, d, a, a, a, 64, a, 64, a, 1 << 50)
    refused("dx_stride", b.tide_ce_grad, desc(), a, a, a, far, a, 64, a, 1 << 50)
    refused("dweight_stride", b.tide_ce_grad, desc(), a, a, a, 64, a, far, a, 1 << 50)


def test_the_status_is_read_next_to_the_operators(graphs):
    import all_gather_gb300 as tide
    assert tide.device_status is graphs.ops.device_status
