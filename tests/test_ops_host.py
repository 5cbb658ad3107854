"""Host checks of the training-step operators, no GPU needed: the C entry
points refuse bad arguments before they touch the device, with the documented
status, the wrappers refuse tensors of the wrong kind, and the 64-bit
reference forms that the GPU tests use agree with differences."""
import ctypes
import re

import pytest
import torch

import ops_reference as ref

A = 0x7F0000000000  # an address that is never read


@pytest.fixture(scope="module")
def tide():
    from all_gather_gb300 import build
    build.build()
    import all_gather_gb300
    all_gather_gb300.load_library()
    return all_gather_gb300


@pytest.fixture(scope="module")
def b(tide):
    from all_gather_gb300 import _binding
    return _binding


def refused(tide, status, match, f, *a):
    with pytest.raises(tide.TideError) as e:
        f(*a)
    assert e.value.status == status, e.value
    assert re.search(match, e.value.detail), e.value.detail


def qk(b, **kw):
    d = dict(tokens=4, q_heads=2, k_heads=1, head_dim=64, rotary_dim=64, max_position=10, table=A, positions=A,
             position_bytes=8, dtype=0, interleaved=0, eps=1e-6, q_weight=A, k_weight=A)
    d.update(kw)
    return b.QkDesc(**d)


def heads(b, p=A, st=128, sh=64):
    return b.Heads(p, st, sh)


@pytest.mark.parametrize("kw, status, match", [
    (dict(tokens=-1), 1, "tokens"), (dict(q_heads=-1), 1, "q_heads"), (dict(k_heads=1 << 21), 1, "k_heads"),
    (dict(head_dim=0), 1, "head_dim"), (dict(head_dim=4097), 1, "head_dim"), (dict(rotary_dim=63), 1, "rotary_dim"),
    (dict(rotary_dim=66), 1, "rotary_dim"), (dict(eps=-1.0), 1, "eps"), (dict(eps=float("nan")), 1, "eps"),
    (dict(dtype=2), 3, "dtype"), (dict(position_bytes=2), 1, "position_bytes"), (dict(table=None), 1, "table"),
    (dict(positions=None), 1, "positions"), (dict(max_position=0), 1, "max_position"), (dict(table=A + 2), 2, "table"),
    (dict(positions=A + 4), 2, "positions"), (dict(q_weight=A + 1), 2, "weight"), (dict(tokens=1 << 50), 1, "tokens"),
])
def test_qk_descriptor_refusals(tide, b, kw, status, match):
    h = heads(b)
    refused(tide, status, match, b.tide_qk_norm_rope, qk(b, **kw), h, h, h, h)
    refused(tide, status, match, b.tide_qk_norm_rope_grad, qk(b, **kw), h, h, h, h, h, h, A, A, A, 1 << 30)
    refused(tide, 1, match, b.tide_qk_norm_rope_grad_workspace, qk(b, **kw))


def test_qk_tensor_refusals(tide, b):
    ok, f = heads(b), b.tide_qk_norm_rope
    none = b.Heads(None, 128, 64)
    for at, name in enumerate(("q", "k", "q_out", "k_out")):
        def call(bad):
            a = [ok] * 4
            a[at] = bad
            return (qk(b), *a)
        refused(tide, 1, f"{name} is NULL", f, *call(none))
        refused(tide, 1, f"{name} is NULL", f, *call(None))
        refused(tide, 2, name, f, *call(heads(b, A + 1)))
        refused(tide, 1, f"{name} has bad strides", f, *call(heads(b, st=-128)))
    refused(tide, 1, "q_out overlap", f, qk(b), ok, ok, heads(b, st=64, sh=64), ok)
    refused(tide, 1, "q_out overlap", f, qk(b), ok, ok, heads(b, st=0, sh=64), ok)
    refused(tide, 1, "q_out overlap", f, qk(b), ok, ok, heads(b, st=128, sh=32), ok)
    g = b.tide_qk_norm_rope_grad
    refused(tide, 1, "gradient goes with", g, qk(b), ok, ok, ok, ok, ok, ok, 0, A, A, 1 << 30)
    refused(tide, 1, "gradient goes with", g, qk(b, k_weight=None), ok, ok, ok, ok, ok, ok, A, A, A, 1 << 30)
    refused(tide, 2, "gradient", g, qk(b), ok, ok, ok, ok, ok, ok, A + 1, A, A, 1 << 30)
    refused(tide, 1, "q is NULL", g, qk(b), ok, ok, None, ok, ok, ok, A, A, A, 1 << 30)
    refused(tide, 1, "workspace", g, qk(b), ok, ok, ok, ok, ok, ok, A, A, A, 16)
    refused(tide, 1, "workspace", g, qk(b), ok, ok, ok, ok, ok, ok, A, A, 0, 1 << 30)
    refused(tide, 2, "workspace", g, qk(b), ok, ok, ok, ok, ok, ok, A, A, A + 16, 1 << 30)


@pytest.mark.parametrize("kw, match", [
    (dict(n=-1), "max_position"), (dict(R=0), "rotary_dim"), (dict(R=7), "rotary_dim"), (dict(base=0.0), "base"),
    (dict(scaling=3), "scaling"), (dict(scaling=1, factor=0.0), "factor"),
    (dict(scaling=2, low=4.0, high=4.0), "factors"), (dict(scaling=2, original=0.0), "factors"),
    (dict(p=0), "table is NULL")])
def test_rope_table_refusals(tide, b, kw, match):
    d = dict(n=10, R=64, base=1e4, scaling=0, factor=8.0, low=1.0, high=4.0, original=8192.0, p=A)
    d.update(kw)
    refused(tide, 1, match, b.tide_rope_table, *d.values())


def ce(b, **kw):
    d = dict(tokens=4, vocab=100, hidden=64, x=A, x_stride=64, weight=A, weight_stride=64, targets=A, target_bytes=8,
             ignore_index=-100)
    d.update(kw)
    return b.CeDesc(**d)


@pytest.mark.parametrize("kw, status, match", [
    (dict(tokens=-1), 1, "tokens"), (dict(tokens=1 << 31), 1, "tokens"), (dict(vocab=0), 1, "vocab"),
    (dict(vocab=1 << 31), 1, "vocab"), (dict(hidden=0), 1, "hidden"), (dict(hidden=(1 << 20) + 1), 1, "hidden"),
    (dict(x_stride=63), 1, "x_stride"), (dict(weight_stride=63), 1, "weight_stride"),
    (dict(target_bytes=1), 1, "target_bytes"), (dict(debug=1), 1, "debug"), (dict(debug=8), 1, "debug"), (dict(x=None), 1, "NULL"), (dict(weight=None), 1, "NULL"),
    (dict(targets=None), 1, "NULL"), (dict(x=A + 1), 2, "aligned"), (dict(weight=A + 1), 2, "aligned"),
    (dict(targets=A + 4), 2, "aligned")])
def test_ce_descriptor_refusals(tide, b, kw, status, match):
    refused(tide, status, match, b.tide_ce_loss, ce(b, **kw), A, A, A, 1 << 40)
    refused(tide, status, match, b.tide_ce_grad, ce(b, **kw), A, A, A, 64, A, 64, A, 1 << 40)


@pytest.mark.parametrize("T, V, H", [(0, 1, 1), (0, 100, 64), (1, 1, 1), (1, 131072, 4096), (70000, 1000, 7), (3, 2000001, 65)])
def test_ce_workspace_sizes(tide, b, T, V, H):
    """Sizes are whole for every shape, no tokens among them, and the gradient's holds a piece of dz and a share of dx."""
    d = ce(b, tokens=T, vocab=V, hidden=H, x_stride=H, weight_stride=H)
    assert 256 <= b.tide_ce_loss_workspace(d) and b.tide_ce_loss_workspace(d) % 256 == 0
    n = b.tide_ce_grad_workspace(d)
    assert n >= 256 and n % 256 == 0 and n >= T * min(V, 8192) * 2 + T * H * 4


def test_ce_tensor_refusals(tide, b):
    f, g = b.tide_ce_loss, b.tide_ce_grad
    refused(tide, 1, "loss or lse is NULL", f, ce(b), 0, A, A, 1 << 40)
    refused(tide, 1, "loss or lse is NULL", f, ce(b), A, 0, A, 1 << 40)
    refused(tide, 2, "loss", f, ce(b), A + 2, A, A, 1 << 40)
    refused(tide, 1, "workspace", f, ce(b), A, A, A, 16)
    refused(tide, 2, "workspace", f, ce(b), A, A, A + 8, 1 << 40)
    for at in (1, 2, 3, 5):
        a = [ce(b), A, A, A, 64, A, 64, A, 1 << 40]
        a[at] = 0
        refused(tide, 1, "is NULL", g, *a)
        a[at] = A + 1
        refused(tide, 2, "aligned", g, *a)
    refused(tide, 1, "dx_stride", g, ce(b), A, A, A, 63, A, 64, A, 1 << 40)
    refused(tide, 1, "dweight_stride", g, ce(b), A, A, A, 64, A, 63, A, 1 << 40)
    refused(tide, 1, "workspace", g, ce(b), A, A, A, 64, A, 64, A, 16)
    refused(tide, 2, "workspace", g, ce(b), A, A, A, 64, A, 64, A + 8, 1 << 40)
    assert b.load_library().tide_ce_loss_workspace(None) == -1
    assert b.load_library().tide_ce_grad_workspace(None) == -1


def test_swiglu_refusals(tide, b):
    ck = b.Ckpt8Desc(A, A, A, A)
    f, g = b.tide_swiglu_ckpt8, b.tide_swiglu_ckpt8_grad
    fwd = lambda **kw: [{**dict(rows=4, cols=64, dt=0, gate=A, gs=64, up=A, us=64, h=A, hs=64, ck=ck), **kw}[k]  # noqa
                        for k in ("rows", "cols", "dt", "gate", "gs", "up", "us", "h", "hs", "ck")]
    bwd = lambda **kw: [{**dict(rows=4, cols=64, dt=0, ck=ck, dh=A, ds=64, dg=A, gs=64, du=A, us=64, h=A, hs=64),  # noqa
                         **kw}[k] for k in ("rows", "cols", "dt", "ck", "dh", "ds", "dg", "gs", "du", "us", "h", "hs")]
    for call, args in ((f, fwd), (g, bwd)):
        refused(tide, 1, "rows", call, *args(rows=-1))
        refused(tide, 1, "cols", call, *args(cols=-1))
        refused(tide, 1, "rows", call, *args(rows=1 << 40, cols=1 << 30))
        refused(tide, 3, "dtype", call, *args(dt=2))
        refused(tide, 1, "checkpoint", call, *args(ck=b.Ckpt8Desc(A, None, A, A)))
        refused(tide, 1, "checkpoint", call, *args(ck=None))
    refused(tide, 1, "gate is NULL", f, *fwd(gate=0))
    refused(tide, 1, "up has row stride", f, *fwd(us=-1))
    refused(tide, 2, "h is not aligned", f, *fwd(h=A + 1))
    refused(tide, 1, "h has row stride", f, *fwd(hs=63))
    refused(tide, 1, "dh is NULL", g, *bwd(dh=0))
    refused(tide, 1, "dgate has row stride", g, *bwd(gs=10))
    refused(tide, 2, "dup is not aligned", g, *bwd(du=A + 1))
    refused(tide, 1, "h has row stride", g, *bwd(hs=10))
    assert b.load_library().tide_swiglu_ckpt8(0, 64, 0, None, 0, None, 0, None, 0, None, None) == 0


def test_wrappers_refuse_the_wrong_kind_of_tensor(tide):
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    y = torch.zeros(4, dtype=torch.int64)
    q = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        tide.linear_cross_entropy(x, x, y)
    with pytest.raises(TypeError, match="bfloat16"):
        tide.linear_cross_entropy(x.float(), x, y)
    with pytest.raises(ValueError, match="CUDA"):
        tide.swiglu_ckpt8(x, x)
    with pytest.raises(TypeError, match="float16"):
        tide.swiglu_ckpt8(x.half(), x.half())
    with pytest.raises(ValueError, match="CUDA"):
        tide.qk_norm_rope(q, q)
    with pytest.raises(ValueError, match="tokens, heads"):
        tide.qk_norm_rope(x, x)
    with pytest.raises(ValueError, match="contiguous"):
        tide.qk_norm_rope(q.transpose(1, 2), q)
    with pytest.raises(ValueError, match="scaling"):
        tide.rope_table(10, 64, scaling="cubic")


def test_structs_have_the_header_s_layout(b):
    assert ctypes.sizeof(b.Heads) == 24 and ctypes.sizeof(b.Ckpt8Desc) == 32
    assert ctypes.sizeof(b.QkDesc) == 8 + 16 + 8 + 16 + 16 + 16 and b.QkDesc.table.offset == 32
    assert ctypes.sizeof(b.CeDesc) == 88 and b.CeDesc.ignore_index.offset == 72


def test_packed_structs_have_the_same_bytes(b):
    p = b.PackedCalls
    assert p.heads(A, 128, 64) == bytes(b.Heads(A, 128, 64))
    assert p.ckpt8(A, A + 1, A + 2, A + 3) == bytes(b.Ckpt8Desc(A, A + 1, A + 2, A + 3))
    v = (7, 2, 1, 64, 32, 10, A, A + 8, 8, 1, 1, 1e-6, A + 16, 0)
    assert p.qk(*v) == bytes(b.QkDesc(*v))


def test_reference_gradients_against_differences():
    """The reference's own gradients, by central differences in 64 bits (error about h^2)."""
    torch.manual_seed(0)
    h = 1e-6
    T, H, D, R = 3, 2, 12, 8
    a = torch.rand(20, R // 2, dtype=torch.float64) * 6
    table, pos = torch.cat((a.cos(), a.sin()), 1), torch.tensor([3, 0, 19])
    x, w, d, vx, vw = (torch.randn(s, dtype=torch.float64) for s in ((T, H, D), (D,), (T, H, D), (T, H, D), (D,)))
    for il in (False, True):
        M = ref.rotation(table, pos, D, il)
        dx, dw, _ = ref.qk_backward(d, x, w, M, 1e-5)
        f = lambda e: (ref.qk_forward(x + e * vx, w + e * vw, M, 1e-5) * d).sum()  # noqa: E731
        assert torch.isclose((f(h) - f(-h)) / (2 * h), (dx * vx).sum() + (dw * vw).sum(), rtol=1e-7)
    x, w, y = torch.randn(5, 6, dtype=torch.float64), torch.randn(9, 6, dtype=torch.float64), torch.tensor([0, 8, -100, 3, 3])
    dl, vx, vw = torch.rand(5, dtype=torch.float64), torch.randn(5, 6, dtype=torch.float64), torch.randn(9, 6, dtype=torch.float64)
    dx, dw, _, _ = ref.ce_grad(x, w, y, ref.ce_loss(x, w, y)[1], dl)
    f = lambda e: (ref.ce_loss(x + e * vx, w + e * vw, y)[0] * dl).sum()  # noqa: E731
    assert torch.isclose((f(h) - f(-h)) / (2 * h), (dx * vx).sum() + (dw * vw).sum(), rtol=1e-7)
    g, u, dh, vg, vu = (torch.randn(4, 7, dtype=torch.float64) for _ in range(5))
    dg, du, _ = ref.swiglu_grad(g, u, dh)
    f = lambda e: (ref.swiglu(g + e * vg, u + e * vu) * dh).sum()  # noqa: E731
    assert torch.isclose((f(h) - f(-h)) / (2 * h), (dg * vg).sum() + (du * vu).sum(), rtol=1e-7)


def test_reference_codes_against_torch():
    """The reference's e4m3 rounding agrees with torch's conversion where no scale is needed."""
    v = ref.e4m3_values()
    assert torch.equal(torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double(), v)
    x = torch.randn(3, 200) * 300
    x[:, 0], x[:, 128] = 448.0, 300.0
    x = x.clamp(-448, 448)
    q, e = ref.encode(x)
    assert (e == 127).all()
    assert torch.equal(q, x.to(torch.float8_e4m3fn).double())
