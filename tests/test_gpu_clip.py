"""ob_tensor_norms, ob_clip_grads, GradClip and OneBitAdam's max_norm on the GPU against the formulas in 64 bits.

Tolerances: a norm's squares and sums are in double (relative error below 1e-9 for these sizes) and it is rounded to fp32
once: 2^-24 of it.  A clipped gradient is widen(g) times a factor that is rounded once and formed from that norm (2^-24
each), the product rounded once (2^-24), then rounded to its type (eps / 2).
"""
import math

import pytest
import torch

import adam_ob_compress_amd as ob

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = 2.0 ** -24


def gradients(sizes, dtype, seed=0, packed=False, scale=1e-2):
    gen = torch.Generator("cuda").manual_seed(seed)
    if packed:   # behind each other without gaps, from the second element on
        flat = (torch.randn(sum(sizes) + 1, generator=gen, device="cuda") * scale).to(dtype)
        out, at = [], 1
        for s in sizes:
            out.append(flat[at:at + s])
            at += s
        return out
    return [(torch.randn(s, generator=gen, device="cuda") * scale * (1 + j % 5)).to(dtype) for j, s in enumerate(sizes)]


def norms_of(grads, kind):
    each = [0.0 if g is None or g.numel() == 0 else float(g.double().abs().max() if kind == "max" else g.double().pow(2).sum().sqrt())
            for g in grads]
    return each + [max(each) if kind == "max" else math.sqrt(sum(x * x for x in each))]


def factor(norm, max_norm, mult):
    return mult * (min(1.0, max_norm / (norm + 1e-6)) if 0 < max_norm < math.inf else 1.0)


SIZES = [[1], [5, 1, 7], [4096, 1, 4095, 1023] * 5, [4097, 5], [1030] * 32, [9] * 33, [20_011, 3, 4096, 1025], [300_007, 16384, 16385, 2], [70_000] * 70, [3] * 500]


@pytest.mark.parametrize("kind", ["2", "max"])
@pytest.mark.parametrize("g", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
def test_norms_and_clipping(sizes, g, kind):
    for packed in (False, True):
        grads = gradients(sizes, DT[g], len(sizes), packed)
        grads = [None if j % 7 == 5 else x for j, x in enumerate(grads)]
        want = norms_of(grads, kind)
        for out in ("f32", "bf16", "f16"):
            l = ob.ob_tensors_create(sizes, DT[g], DT[out])
            norms = torch.full((len(sizes) + 1,), -1.0, device="cuda")
            ob.ob_tensor_norms(l, grads, norms, g_mult=0.5, kind=ob.OB_NORM_MAX if kind == "max" else ob.OB_NORM_2)
            for x, w in zip(norms.tolist(), want):
                assert abs(x - 0.5 * w) <= 1.01 * U * 0.5 * w
            for each in (False, True):
                for max_norm in (want[-1] * 0.1, want[-1] * 10, 0.0, math.inf):
                    outs = [torch.full_like(x, 7.0, dtype=DT[out]) if x is not None else None for x in grads]
                    ob.ob_clip_grads(l, grads, norms, max_norm, g_mult=0.5, out=outs, per_tensor=each)
                    for j, (x, y) in enumerate(zip(grads, outs)):
                        if x is None:
                            continue
                        f = factor(0.5 * want[j if each else -1], max_norm, 0.5)
                        w = x.double() * f
                        assert ((y.double() - w).abs() <= (4 * U + torch.finfo(DT[out]).eps / 2) * w.abs() + torch.finfo(DT[out]).tiny).all()
            if len(sizes) > 60:
                break


@pytest.mark.parametrize("g", ["f32", "bf16"])
def test_in_place(g):
    sizes = [1000, 1, 5000, 77]
    grads = gradients(sizes, DT[g], 3)
    before = [x.clone() for x in grads]
    l = ob.ob_tensors_create(sizes, DT[g], torch.float16)   # in place the list's parameter types do not matter
    norms = torch.zeros(5, device="cuda")
    ob.ob_tensor_norms(l, grads, norms)
    total = norms_of(before, "2")[-1]
    ob.ob_clip_grads(l, grads, norms, total * 2)            # nothing to clip: the same bits
    assert all(torch.equal(x, y) for x, y in zip(grads, before))
    outs = [torch.empty_like(x) for x in grads]
    same = ob.ob_tensors_create(sizes, DT[g], DT[g])
    ob.ob_clip_grads(same, grads, norms, total / 3, out=outs)
    ob.ob_clip_grads(l, grads, norms, total / 3)
    assert all(torch.equal(x, y) for x, y in zip(grads, outs))
    ob.ob_clip_grads(same, grads, norms, total / 3, out=grads)   # out may be the gradients
    ob.ob_clip_grads(same, outs, norms, total / 3, out=outs)
    assert all(torch.equal(x, y) for x, y in zip(grads, outs))


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("kind", [ob.OB_NORM_2, ob.OB_NORM_MAX])
def test_not_finite(kind, bad):
    sizes = [100, 5000, 3]
    for each in (False, True):
        grads = gradients(sizes, torch.float32, 9)
        before = [x.clone() for x in grads]
        grads[1][4097] = bad
        l = ob.ob_tensors_create(sizes, torch.float32, torch.float32)
        norms = torch.zeros(4, device="cuda")
        ob.ob_tensor_norms(l, grads, norms, kind=kind)
        assert norms[[0, 2]].isfinite().all() and not norms[[1, 3]].isfinite().any()
        assert bool(norms[1].isnan()) == math.isnan(bad)
        ob.ob_clip_grads(l, grads, norms, 1e9, per_tensor=each)
        assert grads[1].isnan().all()
        for j in (0, 2):
            assert torch.equal(grads[j], before[j]) if each else bool(grads[j].isnan().all())


def test_empty_lists_and_tensors():
    norms = torch.ones(1, device="cuda")
    l = ob.ob_tensors_create([], torch.float32, torch.float32)
    ob.ob_tensor_norms(l, [], norms)
    ob.ob_clip_grads(l, [], norms, 1.0)
    assert norms.tolist() == [0.0]
    for T in (3, 90):
        norms = torch.ones(T + 1, device="cuda")
        l = ob.ob_tensors_create([0] * T, torch.float32, torch.float32)
        ob.ob_tensor_norms(l, [torch.zeros(0, device="cuda")] * T, norms)
        assert norms.tolist() == [0.0] * (T + 1)
        norms.fill_(1)
        l = ob.ob_tensors_create([5] * T, torch.float32, torch.float32)
        ob.ob_tensor_norms(l, [None] * T, norms)
        assert norms.tolist() == [0.0] * (T + 1)


def test_mixed_types_and_many_launches():
    """Types in turn, more tensors than a launch takes, and sums that do not depend on the call."""
    T = 1000
    sizes = [17 + 5 * (j % 40) for j in range(T)]
    types = [(torch.float32, torch.bfloat16, torch.float16)[j % 3] for j in range(T)]
    grads = [torch.randn(s, generator=torch.Generator("cuda").manual_seed(j), device="cuda").to(d) for j, (s, d) in enumerate(zip(sizes, types))]
    l = ob.ob_tensors_create(sizes, types, types[::-1])
    norms = torch.zeros(T + 1, device="cuda")
    ob.ob_tensor_norms(l, grads, norms)
    for x, w in zip(norms.tolist(), norms_of(grads, "2")):
        assert abs(x - w) <= 1.01 * U * w
    again = torch.zeros_like(norms)
    ob.ob_tensor_norms(l, grads, again, workspace=torch.full((l.norm_bytes,), 255, dtype=torch.uint8, device="cuda"))
    assert torch.equal(norms, again)
    outs = [torch.empty(s, device="cuda", dtype=d) for s, d in zip(sizes, types[::-1])]
    ob.ob_clip_grads(l, grads, norms, 1.0, out=outs)
    f = factor(norms_of(grads, "2")[-1], 1.0, 1.0)
    for x, y in zip(grads, outs):
        w = x.double() * f
        assert ((y.double() - w).abs() <= (4 * U + torch.finfo(y.dtype).eps / 2) * w.abs() + torch.finfo(y.dtype).tiny).all()


def test_long_list():
    """More bytes than the last-level cache keeps, one tensor with more items than a work group has threads."""
    sizes = [3, 400_000_001, 1000]
    grads = gradients(sizes, torch.bfloat16, 1)
    want = norms_of(grads, "2")
    l = ob.ob_tensors_create(sizes, torch.bfloat16, torch.bfloat16)
    norms = torch.zeros(4, device="cuda")
    ob.ob_tensor_norms(l, grads, norms)
    for x, w in zip(norms.tolist(), want):
        assert abs(x - w) <= 1.01 * U * w
    before = grads[1][-70_000:].clone()
    ob.ob_clip_grads(l, grads, norms, 0.25)
    w = before.double() * factor(want[-1], 0.25, 1.0)
    assert ((grads[1][-70_000:].double() - w).abs() <= (4 * U + 2.0 ** -8) * w.abs()).all()
    ob.ob_tensor_norms(l, grads, norms)
    assert abs(float(norms[-1]) - 0.25) <= 0.25 * 2.0 ** -8   # every element is off by at most half a step


def test_graph_and_streams():
    sizes = [5000, 37, 70_001]
    l = ob.ob_tensors_create(sizes, torch.float32, torch.float32)
    grads = gradients(sizes, torch.float32, 5)
    norms, other = torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda")
    outs, want = [torch.empty_like(x) for x in grads], [torch.empty_like(x) for x in grads]
    work = torch.empty(l.norm_bytes, dtype=torch.uint8, device="cuda")

    def both(n, o, w=None, stream=None):
        ob.ob_tensor_norms(l, grads, n, workspace=w, stream=stream)
        ob.ob_clip_grads(l, grads, n, 0.5, out=o, stream=stream)

    both(norms, outs, work)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both(other, want, None, side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(norms, other) and all(torch.equal(x, y) for x, y in zip(outs, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both(norms, outs, work)
    for k in range(3):
        grads[0].mul_(3.0)
        g.replay()
        both(other, want)
        torch.cuda.synchronize()
        assert torch.equal(norms, other) and all(torch.equal(x, y) for x, y in zip(outs, want)), k


def test_refusals():
    l = ob.ob_tensors_create([8, 4], torch.float32, torch.bfloat16)
    g = [torch.ones(8, device="cuda"), torch.ones(4, device="cuda")]
    norms = torch.zeros(3, device="cuda")
    with pytest.raises(ValueError, match="elements"):
        ob.ob_tensor_norms(l, g, norms[:2])
    with pytest.raises(TypeError, match="norms"):
        ob.ob_tensor_norms(l, g, norms.double())
    with pytest.raises(ValueError, match="bytes"):
        ob.ob_tensor_norms(l, g, norms, workspace=torch.zeros(4, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError, match="workspace"):
        ob.ob_tensor_norms(l, g, norms, workspace=torch.zeros(400, device="cuda"))
    with pytest.raises(ob.ObError):
        ob.ob_tensor_norms(l, g, norms, kind=3)
    with pytest.raises(ob.ObError):
        ob.ob_tensor_norms(l, g, norms, g_mult=0.0)
    with pytest.raises(TypeError, match="grads"):
        ob.ob_tensor_norms(l, [g[0].half(), g[1]], norms)
    with pytest.raises(TypeError, match=r"out\[0\]"):
        ob.ob_clip_grads(l, g, norms, 1.0, out=g)
    with pytest.raises(TypeError, match=r"out\[1\]"):
        ob.ob_clip_grads(l, g, norms, 1.0, out=[g[0].bfloat16(), None])
    with pytest.raises(ob.ObError):
        ob.ob_clip_grads(l, g, norms, float("nan"))
    with pytest.raises(ob.ObError):   # one gradient twice, in place
        two = ob.ob_tensors_create([4, 4], torch.float32, torch.float32)
        ob.ob_clip_grads(two, [g[1], g[1]], norms, 1.0)
    with pytest.raises(ValueError, match="contiguous"):
        ob.ob_clip_grads(l, [torch.ones(16, device="cuda")[::2], g[1]], norms, 1.0)
    assert g[0].eq(1).all() and g[1].eq(1).all() and not norms.any()


def test_gradclip_before_two_optimizers():
    """One norm over what Muon and AdamW step; a step whose norm is not finite is left out by both."""
    gen = torch.Generator("cuda").manual_seed(0)
    params = [torch.nn.Parameter(torch.randn(*s, generator=gen, device="cuda") * 0.02) for s in ((48, 40), (48,), (40, 16), (16,))]
    matrices, rest = [p for p in params if p.dim() == 2], [p for p in params if p.dim() < 2]
    clip = ob.GradClip(params, max_norm=1.0)
    opts = [ob.Muon(matrices, lr=1e-3, max_norm=math.inf), ob.AdamW(rest, lr=1e-3, max_norm=math.inf)]
    x = torch.randn(64, 40, generator=gen, device="cuda")

    def backward(scale):
        for p in params:
            p.grad = None
        (((x @ params[0].t() + params[1])[:, :40] @ params[2] + params[3]).square().sum() * scale).backward()

    for scale in (1e-3, 1e3):
        backward(scale)
        want = norms_of([p.grad for p in params], "2")[-1]
        before = [p.grad.clone() for p in params]
        norm = clip()
        assert abs(float(norm) - want) <= 1.01 * U * want
        f = factor(want, 1.0, 1.0)
        for p, b in zip(params, before):
            assert ((p.grad.double() - b.double() * f).abs() <= 4 * U * (b.double() * f).abs()).all()
        for o in opts:
            o.step()
    kept = [p.detach().clone() for p in params]
    backward(1.0)
    params[3].grad[2] = float("inf")
    clip()
    for o in opts:
        o.step()
    assert all(torch.equal(p, k) for p, k in zip(params, kept))
    assert [o.steps() for o in opts] == [2, 2]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_bit_steps_clip_by_norm(dtype):
    """OneBitAdam(max_norm) is OneBitAdam on a gradient that was clipped before."""
    n = 50_001

    def make(**kw):
        plan = ob.ob_plan_create(n, chunk_size=1 << 14)
        return ob.OneBitAdam(plan, *(torch.zeros(n, device="cuda") for _ in range(4)), lr=1e-3, freeze_step=1, **kw)

    a, b = make(max_norm=0.5), make()
    for k in range(3):
        g = torch.randn(n, generator=torch.Generator("cuda").manual_seed(k), device="cuda").to(DT[dtype])
        want = norms_of([g], "2")[0]
        clipped = g.clone()
        l = ob.ob_tensors_create([n], DT[dtype], DT[dtype])
        norms = torch.zeros(2, device="cuda")
        ob.ob_tensor_norms(l, [clipped], norms)
        ob.ob_clip_grads(l, [clipped], norms, 0.5)
        assert a.step(g) == b.step(clipped)
        assert abs(float(a.norm) - want) <= 1.01 * U * want and torch.equal(g, clipped)
        for x, y in ((a.p, b.p), (a.m, b.m), (a.v, b.v), (a.err, b.err)):
            assert torch.equal(x, y)
