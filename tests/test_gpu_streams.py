"""Calls on a stream that is not the current one, without anything between the two that orders them."""
import pytest
import torch

import adam_ob_compress_amd as ob

pytestmark = pytest.mark.gpu


def busy(x):
    """Some milliseconds of work on the current stream."""
    for _ in range(8):
        torch.mm(x, x, out=x.clone())


def test_norms_take_no_memory_that_the_current_stream_still_reads():
    sizes = [70_000] * 70
    l = ob.ob_tensors_create(sizes, torch.float32, torch.float32)
    grads = [torch.full((n,), 0.5, device="cuda") for n in sizes]
    norms, side = torch.zeros(71, device="cuda"), torch.cuda.Stream()
    big = torch.zeros(8192, 8192, device="cuda")
    for _ in range(3):
        x, y = (torch.full((l.norm_bytes,), v, dtype=torch.uint8, device="cuda") for v in (7, 0))
        busy(big)
        torch.cuda.synchronize()
        busy(big)
        y.copy_(x)
        del x   # its memory may be given out again, in the order of this stream
        ob.ob_tensor_norms(l, grads, norms, stream=side)
        torch.cuda.synchronize()
        assert bool((y == 7).all())
        assert norms[0] == float(torch.tensor(0.5 * 70_000 ** 0.5)) and norms[70] == float(torch.tensor(0.5 * 4_900_000 ** 0.5))
