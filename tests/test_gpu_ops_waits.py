"""A bounded device-side wait of the cross entropy that runs out: what it kept from being computed is NaN, the rest is
right, and the status says so.  Nothing hangs: a fill is left out and the waits end after 50 ms."""
import pytest
import torch

from test_gpu_ops import BF16, ce_inputs, tide  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

# A pair of blocks loses its first tile and the ones after it: one tile of few; one of many on all pairs; a pair with
# several tiles; several pieces and shares of the vocabulary.
SIZES = [(300, 2000, 128), (7, 300, 64), (1500, 9000, 64), (600, 50001, 200)]


def kept(got, want):
    """Every element is NaN or what it should be; how many are NaN."""
    lost = torch.isnan(got) & ~torch.isnan(want)
    assert torch.equal(got[~lost], want[~lost])
    return int(lost.sum())


@pytest.mark.parametrize("T, V, H", SIZES)
@pytest.mark.parametrize("grad", [False, True])
def test_what_a_lost_wait_leaves(tide, T, V, H, grad):
    from all_gather_gb300 import _binding as b
    x, w, y = ce_inputs(T, T, V, H)
    loss, lse = tide.linear_cross_entropy(x, w, y)
    d = torch.rand(T, device="cuda")
    want = tide.linear_cross_entropy_grad(x, w, y, lse, d) if grad else (loss, lse)
    assert tide.ops.device_status() == tide.TIDE_OK
    desc = tide.ops._ce_desc(x, w, y, -100)[0]
    desc.debug = tide.TIDE_DEBUG_SHORT_WAIT | tide.TIDE_DEBUG_SKIP_FILL
    got = [torch.full_like(t, 5) for t in want]
    n = (b.tide_ce_grad_workspace if grad else b.tide_ce_loss_workspace)(desc)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    p = [t.data_ptr() for t in (*got, ws)]
    stream = torch.cuda.current_stream().cuda_stream
    if grad:
        b.tide_ce_grad(desc, lse.data_ptr(), d.data_ptr(), p[0], H, p[1], H, p[2], n, stream)
    else:
        b.tide_ce_loss(desc, p[0], p[1], p[2], n, stream)
    assert tide.ops.device_status() == tide.TIDE_ERR_TIMEOUT
    assert tide.ops.device_status() == tide.TIDE_OK
    for a, c in zip(got, want):
        assert kept(a, c) > 0
    again = tide.linear_cross_entropy_grad(x, w, y, lse, d) if grad else tide.linear_cross_entropy(x, w, y)
    assert all(torch.equal(a, c) for a, c in zip(again, want))
    assert tide.ops.device_status() == tide.TIDE_OK
