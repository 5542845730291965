"""The Muon step on matrices beyond a compute unit's LDS: the launches that large matrices take, in all that a call can ask for.

Tolerances: those of test_gpu_muon.py, whose bounds are used here.
"""
import math

import pytest
import torch

import adam_ob_compress_amd as ob
from test_gpu_muon import U, element_bound, exact

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols,iterations", [(64, 17_000_000, 2), (17_000_000, 64, 2), (1, 150_000_000, 1)])
def test_longest_matrices(rows, cols, iterations):
    """Next to the longest that a plan takes.  All but some columns (of the smaller side) are zeros, spread over the whole length, its
    ends among them: zeros add no error to a sum, so the bounds are those of the matrix without them."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    side, length = min(rows, cols), max(rows, cols)
    gen = torch.Generator("cuda").manual_seed(side)
    at = torch.randint(0, length, (1500,), generator=gen, device="cuda")
    at = torch.cat([at, torch.arange(70, device="cuda"), length - 1 - torch.arange(70, device="cuda")]).unique()
    some = (torch.randn(side, at.numel(), generator=gen, device="cuda") * torch.linspace(0.2, 2, side, device="cuda")[:, None]).bfloat16()
    g = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    (g.t() if rows > cols else g)[:, at] = some
    p = torch.zeros_like(g)
    l = ob.ob_tensors_create([g.numel()], torch.bfloat16, torch.bfloat16)
    plan = ob.ob_muon_create(l, [g.shape])
    m = torch.zeros(l.state_elems, device="cuda")
    work = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    ob.ob_muon_step(plan, [g], [p], m, ob.muon_hparams(lr=1.0, momentum=0.0, weight_decay=0.0, iterations=iterations,
                                                      scale=ob.OB_MUON_PLAIN), work)
    p = p.t() if rows > cols else p
    got, want, bound = p[:, at].double(), exact(some, iterations), element_bound(some, iterations)
    assert ((got + want).abs() <= bound + (2.0 ** -8 + 4 * U) * (want.abs() + bound)).all()
    p[:, at] = 0
    assert not p.any()   # nothing but the decay, which is 0, where there is no gradient


def test_longer_matrices_are_refused():
    for shape in ((64, 17_100_000), (17_100_000, 64), (8, 160_000_000)):
        l = ob.ob_tensors_create([math.prod(shape)], torch.bfloat16, torch.bfloat16)
        with pytest.raises(ob.ObError):
            ob.ob_muon_create(l, [shape])
