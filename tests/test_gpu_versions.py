"""Calls that overwrite tensors raise their version, so that autograd refuses a backward pass that needs what was there."""
import pytest
import torch

import adam_ob_compress_amd as ob

pytestmark = pytest.mark.gpu


def saved(x):
    """A result whose backward pass needs x as it is now."""
    return (torch.ones(x.shape, device="cuda", requires_grad=True) * x.detach()).sum()


def overwrites(call, *tensors):
    """The call raises each tensor's version, and a backward pass that needs one of them is refused."""
    results, before = [saved(x) for x in tensors], [x._version for x in tensors]
    call()
    for x, y, v in zip(tensors, results, before):
        assert x._version > v
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()


@pytest.fixture
def lists():
    gen = torch.Generator("cuda").manual_seed(1)
    shapes = [(40, 24), (200, 300), (8, 8)]
    grads, params = ([torch.randn(s, generator=gen, device="cuda") for s in shapes] for _ in range(2))
    return shapes, grads, params, ob.ob_tensors_create([p.numel() for p in params], torch.float32, torch.float32)


def test_matmul():
    a = torch.randn(40, 24, device="cuda").bfloat16()
    out, c = torch.zeros(40, 40, device="cuda"), torch.ones(40, 40, device="cuda")
    overwrites(lambda: ob.ob_matmul(a, a.t(), out), out)
    v = (a._version, c._version)
    overwrites(lambda: ob.ob_matmul(a, a.t(), out, beta=1.0, c=c, stream=torch.cuda.current_stream()), out)
    assert v == (a._version, c._version)
    v = out._version
    with pytest.raises(ob.ObError):
        ob.ob_matmul(a, a.t(), out, alpha=float("inf"))
    assert out._version == v
    with torch.inference_mode():   # tensors without a version
        plain = torch.zeros(40, 40, device="cuda")
    ob.ob_matmul(a, a.t(), plain)
    assert torch.equal(plain, plain.t()) and plain.any()


def test_clipping(lists):
    _, grads, _, l = lists
    norms, outs = torch.zeros(4, device="cuda"), [torch.zeros_like(g) for g in grads]
    overwrites(lambda: ob.ob_tensor_norms(l, grads, norms), norms)
    v = [g._version for g in grads]
    overwrites(lambda: ob.ob_clip_grads(l, grads, norms, 0.1, out=outs), *outs)
    assert v == [g._version for g in grads]
    overwrites(lambda: ob.ob_clip_grads(l, grads, norms, 0.1), *grads)
    v = [g._version for g in grads]
    ob.ob_clip_grads(l, [grads[0], None, grads[2]], norms, 0.1)
    assert [g._version - x for g, x in zip(grads, v)][1] == 0
    params = [torch.nn.Parameter(g.clone()) for g in grads]
    for p in params:
        p.grad = p.detach().clone()
    overwrites(ob.GradClip(params, max_norm=0.1), *[p.grad for p in params])


def test_steps_over_lists(lists):
    shapes, grads, params, l = lists
    m, v = torch.zeros(l.state_elems, device="cuda"), torch.zeros(l.state_elems, device="cuda")
    plan = ob.ob_muon_create(l, shapes)
    work = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    overwrites(lambda: ob.ob_muon_step(plan, grads, params, m, ob.muon_hparams(), work), *params)
    overwrites(lambda: ob.ob_adamw_step(l, grads, params, m, v, ob.adamw_hparams(step=1)), *params)
    codes = [torch.zeros(l.state_elems, dtype=d, device="cuda") for d in (torch.int8, torch.uint8)]
    scales = [torch.zeros(l.state_elems // ob.OB_STATE_BLOCK, device="cuda") for _ in range(2)]
    overwrites(lambda: ob.ob_adamw8_step(l, grads, params, codes[0], scales[0], codes[1], scales[1], ob.adamw_hparams(step=1)), *params)
    before = [p._version for p in params]
    ob.ob_muon_step(plan, [grads[0], None, grads[2]], params, m, ob.muon_hparams(), work)
    assert params[1]._version == before[1] and params[0]._version > before[0]
    for make in (lambda ps: ob.Muon(ps), lambda ps: ob.AdamW(ps), lambda ps: ob.AdamW(ps, state_bits=8, max_norm=1.0)):
        opt = make([torch.nn.Parameter(p.clone()) for p in params])
        overwrites(lambda: opt.step(grads), *opt.params)
