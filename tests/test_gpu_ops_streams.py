"""The operators on a stream that is passed and is not the current one."""
import pytest
import torch

import test_gpu_ops
from test_gpu_ops import BF16, swiglu_inputs, tide  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def all_ops(tide):
    """test_gpu_ops' calls, with inputs that all outlive the call (its SwiGLU gradient copies one for each)."""
    ops = test_gpu_ops.all_ops(tide)
    gate, up = (t.contiguous() for t in swiglu_inputs(93, 40, 300, BF16, "packed"))
    _, ckpt = tide.swiglu_ckpt8(gate, up)
    ops["swiglu_grad"] = lambda s: tide.swiglu_ckpt8_grad(ckpt, up, stream=s)
    return ops


@pytest.mark.parametrize("raw", [False, True])
def test_a_passed_stream_that_is_not_current(tide, raw):
    """Behind work that delays it, and while the current stream fills all the memory that it is handed meanwhile: the
    same bits."""
    ops = all_ops(tide)
    want = {n: [t.clone() for t in f(None)] for n, f in ops.items()}
    side = torch.cuda.Stream()
    here = torch.cuda.current_stream()
    for n, f in ops.items():
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(5_000_000)
        got = f(side.cuda_stream if raw else side)
        assert torch.cuda.current_stream() == here
        filled = [torch.full((size,), 255, dtype=torch.uint8, device="cuda")
                  for size in (256, 4096, 65536, 400_000, 1 << 20, 3 << 20) for _ in range(8)]
        here.synchronize()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[n])), n
        del filled


def test_default_stream_by_its_handle(tide):
    ops = all_ops(tide)
    want = {n: [t.clone() for t in f(None)] for n, f in ops.items()}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = {n: f(0) for n, f in ops.items()}
    torch.cuda.synchronize()
    for n in ops:
        assert all(torch.equal(a, b) for a, b in zip(got[n], want[n])), n
