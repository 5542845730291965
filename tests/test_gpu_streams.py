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


def one_bit(cls, n, freeze_step, **kw):
    plan = ob.ob_plan_create(n, chunk_size=1 << 14)
    gen = torch.Generator("cuda").manual_seed(3)
    state = [torch.randn(n, generator=gen, device="cuda") * 1e-2 for _ in range(4)]
    state[2].square_()
    return cls(plan, *state, lr=1e-3, freeze_step=freeze_step, max_norm=0.5, **kw)


@pytest.mark.parametrize("freeze_step", [0, 1])
@pytest.mark.parametrize("cls", [ob.OneBitAdam, ob.OneBitLamb])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_first_one_bit_step_on_another_stream_and_captured(cls, dtype, freeze_step):
    """With max_norm, a first step that the current stream's work has no order with, and one that is captured."""
    n = 100_003
    g = torch.randn(n, generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(dtype)
    a, b, c = (one_bit(cls, n, freeze_step) for _ in range(3))
    grads = [g.clone() for _ in range(3)]
    side, big = torch.cuda.Stream(), torch.zeros(8192, 8192, device="cuda")
    busy(big)
    torch.cuda.synchronize()
    a.step(grads[0])
    torch.cuda.synchronize()
    busy(big)
    b.step(grads[1], stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.step(grads[2])
    graph.replay()
    torch.cuda.synchronize()
    assert float(a.norm) > 0.5
    for o, x in ((b, grads[1]), (c, grads[2])):
        assert torch.equal(a.norm, o.norm) and torch.equal(grads[0], x)
        for k in ("err", "m", "v", "p", "words", "scales"):
            assert torch.equal(getattr(a, k), getattr(o, k)), k
