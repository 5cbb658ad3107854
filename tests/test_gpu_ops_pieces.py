"""Cross entropy over more than one piece of the vocabulary, and of more tokens than a joining block takes at once.

The gradient keeps dz of one piece at a time: 2^27 elements of it, at least 8192 columns in steps of 256.  Each case
has a last piece that is shorter, and targets on both sides of every border."""
import pytest
import torch

import ops_reference as ref
from test_gpu_ops import BF16, F32, Framed, ce_inputs, close, gen, tide  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def piece(T):
    return max(8192, (1 << 27) // T // 256 * 256)


def inputs(T, V, H, layout):
    x, w, y = ce_inputs(T + V + H, T, V, H, layout)
    borders = [v for b in (*range(0, V, piece(T)), V) for v in (b - 1, b) if 0 <= v < V]
    y[:len(borders) * 3] = torch.tensor(borders * 3, device="cuda")
    return x, w, y


CASES = [
    # T, V, H, layout, pieces
    (16400, 16385, 64, "plain", 3),   # a last piece of one column: fewer steps than shares of the sum
    (16400, 16400, 8, "wide", 3),
    (16400, 20001, 33, "odd", 3),     # odd rows: the weight's copy takes the gradient of pieces that are done
    (1100, 125001, 40, "plain", 2),
    (2500, 53601, 72, "odd", 2),
]


@pytest.mark.parametrize("T, V, H, layout, pieces", CASES)
def test_several_pieces(tide, T, V, H, layout, pieces):
    assert -(-V // piece(T)) == pieces
    x, w, y = inputs(T, V, H, layout)
    loss, lse = tide.linear_cross_entropy(x, w, y)
    wl, ws, bound = ref.ce_loss(x, w, y)
    close(loss, wl, bound, "loss")
    close(lse, ws, bound, "lse")
    lse = ws.float()
    del wl, ws, bound
    dloss = torch.rand(T, generator=gen(T), device="cuda") / T
    pad, shift = {"plain": (0, 0), "wide": (8, 8), "odd": (1, 1)}[layout]
    fx, fw = Framed((T, H), BF16, pad, shift), Framed((V, H), BF16, pad, shift)
    tide.linear_cross_entropy_grad(x, w, y, lse, dloss, out=(fx.t, fw.t))
    fx.check(), fw.check()
    dx, dw, bx, bw = ref.ce_grad(x, w, y, lse, dloss)
    close(fx.t, dx, bx, "dx")
    close(fw.t, dw, bw, "dweight")
    again = tide.linear_cross_entropy_grad(x, w, y, lse, dloss)
    assert torch.equal(again[0], fx.t) and torch.equal(again[1], fw.t)


def test_pieces_do_not_depend_on_what_the_workspace_held(tide):
    x, w, y = inputs(16400, 16500, 24, "plain")
    lse = tide.linear_cross_entropy(x, w, y)[1]
    d = torch.full((16400,), 1e-4, device="cuda")
    want = tide.linear_cross_entropy_grad(x, w, y, lse, d)
    ws = torch.full((1 << 30,), 255, dtype=torch.uint8, device="cuda")
    got = tide.linear_cross_entropy_grad(x, w, y, lse, d, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_pieces_with_a_wait_that_runs_out(tide):
    """What is lost in one piece stays lost in the sum over all, the rest is right."""
    from all_gather_gb300 import _binding as b
    T, V, H = 16400, 16400, 64
    x, w, y = inputs(T, V, H, "plain")
    lse = tide.linear_cross_entropy(x, w, y)[1]
    d = torch.full((T,), 1e-4, device="cuda")
    want = tide.linear_cross_entropy_grad(x, w, y, lse, d)
    desc = tide.ops._ce_desc(x, w, y, -100)[0]
    desc.debug = tide.TIDE_DEBUG_SHORT_WAIT | tide.TIDE_DEBUG_SKIP_FILL
    n = b.tide_ce_grad_workspace(desc)
    ws, dx, dw = torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.empty_like(x), torch.empty_like(w)
    b.tide_ce_grad(desc, lse.data_ptr(), d.data_ptr(), dx.data_ptr(), H, dw.data_ptr(), H, ws.data_ptr(), n,
                   torch.cuda.current_stream().cuda_stream)
    assert tide.ops.device_status() == tide.TIDE_ERR_TIMEOUT
    for got, good in ((dx, want[0]), (dw, want[1])):
        lost = torch.isnan(got)
        assert lost.any() and torch.equal(got[~lost], good[~lost])
