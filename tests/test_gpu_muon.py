"""ob_muon_step and Muon on the GPU against the formulas in 64 bits.

Tolerances.  m: two products and a sum in double, rounded once: 2^-24 of it, and 2^-24 of (1-mu) g' for the scaled gradient.
X: u = 2^-11 is half a step of fp16.  The kernels round X_0, then in each iteration A, B = b A + c A^2 and X to fp16 once (the fp32 sums are
off by K 2^-23 of the sum of magnitudes at most, K the length).  With |.| element by element, dX the error of X on entry:
  dA <= |dX| |X|' + |X| |dX|' + |dX| |dX|' + (u + K 2^-23) (|X| |X|')
  dB <= |b| dA + |c| (dA |A| + |A| dA + dA dA) + u (|b A| + |c A A|) + |c| K 2^-23 |A| |A|
  dX <= a |dX| + dB |X| + |B| |dX| + dB |dX| + u |X'| + K 2^-23 |B| |X|
(what is rounded is within the sums' error of the exact value; u is applied to the magnitudes' bounds, which are not smaller).  Values below
2^-14 in fp16 are spaced 2^-24 apart, which adds 2^-25 over the power of two that a matrix is held times.  That bound holds for one and two
iterations.  For more the errors' growth is bounded by the polynomial f(s) = a s + b s^3 + c s^5 itself: an error E of X (Frobenius
norm) becomes at most L |E|, L = the largest divided difference of f over X's singular values and their negatives (f is
odd; second-order terms add less than |E| 30 |E|), and each iteration adds at most the three roundings' norms.
"""
import math

import pytest
import torch

import adam_ob_compress_amd as ob

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
A, B, C = 3.4445, -4.7750, 2.0315
U, UH = 2.0 ** -24, 2.0 ** -11


def exact(u, iterations, eps=1e-7):
    """X of one matrix in 64 bits, in u's orientation, from the smaller side."""
    x = u.double()
    x = x / (x.square().sum().sqrt() + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    for _ in range(iterations):
        g = x @ x.t()
        x = A * x + (B * g + C * g @ g) @ x
    return x.t() if tall else x


def element_bound(u, iterations, eps=1e-7):
    """Bound of each element's error by the recursion above, in u's orientation."""
    x = u.double()
    x = x / (x.square().sum().sqrt() + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    r, k = x.shape
    sub_x, sub_a = 2.0 ** -25 / 512, 2.0 ** -25 / 1024
    d = (UH + 4 * U) * x.abs() + sub_x
    for _ in range(iterations):
        g = x @ x.t()
        ax, ag = x.abs(), g.abs()
        dg = d @ ax.t() + ax @ d.t() + d @ d.t() + (UH + k * 2 * U) * (ax @ ax.t()) + sub_a
        poly = B * g + C * g @ g
        db = abs(B) * dg + C * (dg @ ag + ag @ dg + dg @ dg) + (UH + 4 * U) * (abs(B) * ag + C * ag @ ag) + C * r * 2 * U * ag @ ag + sub_a
        new = A * x + poly @ x
        d = A * d + db @ ax + poly.abs() @ d + db @ d + (r * 2 * U + 4 * U) * (poly.abs() @ ax + A * ax)
        d = d + UH * (new.abs() + d) + sub_x
        x = new
    return d.t() if tall else d


def norm_bound(u, iterations, eps=1e-7):
    """Bound of the error's Frobenius norm."""
    x = u.double()
    x = x / (x.square().sum().sqrt() + eps)
    x = x.t() if x.shape[0] > x.shape[1] else x
    r, k = x.shape
    s = torch.linalg.svdvals(x)
    sub = 2.0 ** -25 / 512 * math.sqrt(r * k)
    e = (UH + 4 * U) * 1.0 + sub
    for _ in range(iterations):
        both = torch.cat([s, -s])
        f = A * both + B * both ** 3 + C * both ** 5
        gap = both[:, None] - both[None, :]
        slope = (A + 3 * B * both ** 2 + 5 * C * both ** 4)[:, None].expand_as(gap)
        L = float(torch.where(gap.abs() > 1e-6, (f[:, None] - f[None, :]) / torch.where(gap == 0, 1.0, gap), slope).abs().max())
        top, fro = float(s.max()), float(s.square().sum().sqrt())
        a_top, a_fro = top ** 2, float((s ** 4).sum().sqrt())
        b_fro = float(((B * s ** 2 + C * s ** 4) ** 2).sum().sqrt())
        # the sums' errors: K 2^-23 | |X| |X|' |, at most K 2^-23 of the product of the norms
        da = UH * a_fro + k * 2 * U * fro ** 2 + 2.0 ** -25 / 1024 * r
        db = UH * (abs(B) * a_fro + C * a_fro * a_top) + C * r * 2 * U * a_fro ** 2 + 2.0 ** -25 / 1024 * r
        new = (A * s + B * s ** 3 + C * s ** 5).abs()
        local = (da * (abs(B) + 2 * C * a_top) + db) * top + UH * float(new.square().sum().sqrt()) + r * 2 * U * b_fro * fro + sub
        e = (L + 30 * e) * e + local * (1 + 30 * e)
        s = new
    return e


def make(shapes, g="f32", p="f32", seed=0, kind="gauss"):
    gen = torch.Generator("cuda").manual_seed(seed)

    def one(shape):
        x = torch.randn(*shape, generator=gen, device="cuda")
        if kind == "graded":
            x = x * torch.exp(torch.randn(*shape[:-1], 1, generator=gen, device="cuda"))
        return x * 1e-3

    grads = [one(s).to(DT[g]) for s in shapes]
    sizes = [math.prod(s) for s in shapes]
    l = ob.ob_tensors_create(sizes, DT[g], DT[p])
    m = torch.zeros(l.state_elems, device="cuda")
    for j, s in enumerate(shapes):
        m[l.state_offset(j):l.state_offset(j) + sizes[j]] = one(s).view(-1) * 0.3
    params = [torch.randn(*s, generator=gen, device="cuda").mul_(0.02).to(DT[p]) for s in shapes]
    plan = ob.ob_muon_create(l, shapes)
    return l, plan, grads, params, m, torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")


def part(l, flat, t, shape):
    return flat[l.state_offset(t):l.state_offset(t) + math.prod(shape)].view(shape)


def directions(l, shapes, grads, m, mu, nesterov, mult=1.0):
    """The new momentum and u of every tensor, in 64 bits."""
    out = []
    for t, (s, g) in enumerate(zip(shapes, grads)):
        old = part(l, m, t, s).double()
        new = mu * old + (1 - mu) * mult * g.double()
        out.append((new, (1 - mu) * mult * g.double() + mu * new if nesterov else new))
    return out


SHAPES = [[(1, 1)], [(1, 7)], [(8, 8)], [(33, 17)], [(64, 64), (64, 64)], [(100, 37), (5, 129), (129, 5)], [(3, 40, 24), (2, 24, 40)],
          [(130, 300), (300, 130)], [(256, 256), (264, 520)], [(16, 2000)], [(2000, 3)], [(520, 700), (64, 1), (1, 64)],
          [(160, 160), (168, 168)], [(128, 256), (300, 96), (17, 1000)], [(2400, 9), (20, 1500), (32, 32)]]


@pytest.mark.parametrize("iterations", [1, 2])
@pytest.mark.parametrize("shapes", SHAPES, ids=str)
def test_each_element_after_few_iterations(shapes, iterations):
    l, plan, grads, params, m, work = make(shapes, seed=len(shapes))
    mu = float(torch.tensor(0.9))
    want = directions(l, shapes, grads, m, mu, True)
    for p in params:
        p.zero_()
    hp = ob.muon_hparams(lr=1.0, momentum=mu, weight_decay=0.0, iterations=iterations, scale=ob.OB_MUON_PLAIN)
    ob.ob_muon_step(plan, grads, params, m, hp, work)
    for t, (s, (new, u), p) in enumerate(zip(shapes, want, params)):
        assert ((part(l, m, t, s).double() - new).abs() <= 4 * U * new.abs() + 1e-12).all()
        for y, x in zip(p.view(-1, *s[-2:]), u.view(-1, *s[-2:])):
            far = (-y.double() - exact(x, iterations)).abs()
            assert (far <= element_bound(x, iterations) + 4 * U).all(), float((far / element_bound(x, iterations)).max())


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("kind", ["gauss", "graded"])
@pytest.mark.parametrize("shapes", SHAPES + [[(768, 768)], [(512, 1408), (1408, 512)]], ids=str)
def test_five_iterations(shapes, kind, nesterov):
    l, plan, grads, params, m, work = make(shapes, seed=7, kind=kind)
    want = directions(l, shapes, grads, m, float(torch.tensor(0.95)), nesterov)
    for p in params:
        p.zero_()
    hp = ob.muon_hparams(lr=1.0, momentum=0.95, weight_decay=0.0, scale=ob.OB_MUON_PLAIN, nesterov=nesterov)
    ob.ob_muon_step(plan, grads, params, m, hp, work)
    for s, (_, u), p in zip(shapes, want, params):
        for y, x in zip(p.view(-1, *s[-2:]), u.view(-1, *s[-2:])):
            far = float((-y.double() - exact(x, 5)).square().sum().sqrt())
            assert far <= norm_bound(x, 5), (far, norm_bound(x, 5))


@pytest.mark.parametrize("scale", [ob.OB_MUON_PLAIN, ob.OB_MUON_SHAPE, ob.OB_MUON_MATCH_RMS])
@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("g,p", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "f32")])
def test_parameters(g, p, master, scale):
    """Types, master copies, decay and scales: the parameters' line from the X that the same step gives on zero parameters."""
    shapes = [(72, 40), (40, 72), (2, 33, 65), (65, 33)]
    mults = [1.0, 0.5, 2.0, 1.0], [0.0, 1.0, 1.0, 3.0]
    l0, plan, grads, params, m, work = make(shapes, g, "f32", seed=3)
    x = [q.zero_() for q in params]
    ob.ob_muon_step(plan, grads, x, m.clone(), ob.muon_hparams(lr=1.0, weight_decay=0.0, scale=ob.OB_MUON_PLAIN), work)
    l = ob.ob_tensors_create([math.prod(s) for s in shapes], DT[g], DT[p], *mults)
    plan = ob.ob_muon_create(l, shapes)
    gen = torch.Generator("cuda").manual_seed(5)
    old = [torch.randn(*s, generator=gen, device="cuda") * 0.02 for s in shapes]
    params = [o.to(DT[p], copy=True) for o in old]   # the step must not change what it is compared with
    flat = None
    if master:
        flat = torch.zeros(l.state_elems, device="cuda")
        for t, o in enumerate(old):
            part(l, flat, t, o.shape).copy_(o)
    lr, wd = float(torch.tensor(0.01)), float(torch.tensor(0.1))
    ob.ob_muon_step(plan, grads, params, m, ob.muon_hparams(lr=lr, weight_decay=wd, scale=scale), work, master=flat)
    for t, (s, y, o) in enumerate(zip(shapes, x, old)):
        R, K = s[-2:]
        f = {ob.OB_MUON_PLAIN: 1.0, ob.OB_MUON_SHAPE: math.sqrt(max(1.0, R / K)), ob.OB_MUON_MATCH_RMS: 0.2 * math.sqrt(max(R, K))}[scale]
        kept = master and p != "f32"
        start = (o if kept else o.to(DT[p])).double()
        want = start - lr * mults[0][t] * (wd * mults[1][t] * start - f * y.double())
        size = start.abs() + lr * mults[0][t] * (wd * mults[1][t] * start.abs() + f * y.double().abs())
        if kept:
            assert ((part(l, flat, t, s).double() - want).abs() <= 6 * U * size).all()
            assert torch.equal(params[t], part(l, flat, t, s).to(DT[p]))
        else:
            eps = torch.finfo(DT[p]).eps / 2
            assert ((params[t].double() - want).abs() <= (6 * U + eps) * size + torch.finfo(DT[p]).tiny).all()


def test_control_block():
    """Clipping, the rate's factor, steps left out, the count: by ob_grad_norm as for AdamW."""
    shapes = [(48, 32), (16, 64)]
    l, plan, grads, params, m, work = make(shapes)
    start, m0 = [p.clone() for p in params], m.clone()
    ctl = ob.control_create()
    f = ob.control_fields(ctl)
    f["lr_scale"].fill_(0.5)
    hp = ob.muon_hparams(lr=0.02)
    ob.ob_muon_step(plan, grads, params, m, hp, work, control=ctl, norm=(0.25, 1e-3))
    total = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    assert abs(float(f["norm"]) - 0.25 * total) <= 1.01 * U * total and int(f["step"]) == 1
    mult = 0.25 * min(1.0, 1e-3 / (0.25 * total + 1e-6))
    want = directions(l, shapes, grads, m0, 0.95, True, mult)
    for t, (s, (new, _)) in enumerate(zip(shapes, want)):
        assert ((part(l, m, t, s).double() - new).abs() <= 6 * U * (new.abs() + part(l, m0, t, s).double().abs()) + 1e-12).all()
    # the same step with the gradients scaled by hand and half the rate
    again, m1 = [p.clone() for p in start], m0.clone()
    scaled = [g * f["grad_scale"] for g in grads]
    ob.ob_muon_step(plan, scaled, again, m1, ob.muon_hparams(lr=0.01), work)
    assert torch.equal(m, m1) and all(torch.equal(x, y) for x, y in zip(params, again))
    kept, m2 = [p.clone() for p in params], m.clone()
    grads[1][3, 5] = float("nan")
    ob.ob_muon_step(plan, grads, params, m, hp, work, control=ctl, norm=(1.0, 0.0))
    assert torch.equal(m, m2) and all(torch.equal(x, y) for x, y in zip(params, kept))
    assert int(f["step"]) == 1 and int(f["skipped"]) == 1
    # a refused step is not counted
    grads[1][3, 5] = 0.0
    with pytest.raises(ob.ObError):
        ob.ob_muon_step(plan, grads, params, m, ob.muon_hparams(iterations=0), work, control=ctl, norm=(1.0, 0.0))
    assert int(f["step"]) == 1 and int(f["skipped"]) == 1


def test_missing_gradients_zeros_and_bad_values():
    shapes = [(40, 24), (24, 40), (0, 8, 8), (64, 64)]
    l, plan, grads, params, m, work = make(shapes)
    kept, m0 = [p.clone() for p in params], m.clone()
    work.fill_(255)   # of any content: NaN in fp16
    hp = ob.muon_hparams(lr=0.1)
    ob.ob_muon_step(plan, [grads[0], None, grads[2], grads[3]], params, m, hp, work)
    assert torch.equal(params[1], kept[1]) and torch.equal(part(l, m, 1, shapes[1]), part(l, m0, 1, shapes[1]))
    assert params[0].isfinite().all() and not torch.equal(params[0], kept[0]) and not torch.equal(params[3], kept[3])
    ob.ob_muon_step(plan, [None] * 4, params, m, hp, work)
    # a matrix of zeros: its decay alone
    l, plan, grads, params, m, work = make([(40, 24)])
    m.zero_()
    grads[0].zero_()
    old = params[0].clone()
    ob.ob_muon_step(plan, grads, params, m, ob.muon_hparams(lr=0.5, weight_decay=0.5), work)
    assert torch.equal(params[0], torch.addcmul(old, old, torch.tensor(0.5, device="cuda"), value=-0.5))
    # tiny and huge gradients, one spike: finite, and of unit size; a NaN stays in its matrix
    for scale, spike in ((1e-5, False), (1e18, False), (1e-3, True)):
        shapes = [(40, 24), (24, 48)]
        l, plan, grads, params, m, work = make(shapes)
        m.zero_()
        for g, p in zip(grads, params):
            g.mul_(1e3 * scale)
            if spike:
                g[3, 7] = 1e6 * scale
            p.zero_()
        want = [u for _, u in directions(l, shapes, grads, m, float(torch.tensor(0.95)), True)]
        ob.ob_muon_step(plan, grads, params, m, ob.muon_hparams(lr=1.0, weight_decay=0.0, scale=ob.OB_MUON_PLAIN), work)
        for u, p in zip(want, params):
            far = float((-p.double() - exact(u, 5)).square().sum().sqrt())
            assert far <= norm_bound(u, 5)
    grads[0][1, 1] = float("nan")
    before = params[1].clone()
    ob.ob_muon_step(plan, grads, params, m, hp, work)
    assert params[0].isnan().all() and params[1].isfinite().all() and not torch.equal(params[1], before)


def test_mixed_types_many_tensors_and_strides():
    """Types in turn, more tensors than a launch takes, parameters and gradients at any element."""
    T = 430
    shapes = [((9, 16), (24, 8), (8, 11))[j % 3] for j in range(T)]
    types = [("f32", "bf16", "f16")[j % 2] for j in range(T)]
    sizes = [math.prod(s) for s in shapes]
    gen = torch.Generator("cuda").manual_seed(1)
    bucket = {d: torch.randn(sum(sizes) + 1, generator=gen, device="cuda").to(DT[d]) for d in ("f32", "bf16")}
    grads, params, at = [], [], 1
    for s, n, d in zip(shapes, sizes, types):
        grads.append(bucket[d][at:at + n].view(s))
        params.append(torch.zeros(n + 1, device="cuda", dtype=DT[d])[1:].view(s))
        at += n
    l = ob.ob_tensors_create(sizes, [DT[d] for d in types], [DT[d] for d in types])
    plan = ob.ob_muon_create(l, shapes)
    m = torch.zeros(l.state_elems, device="cuda")
    work = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    ob.ob_muon_step(plan, grads, params, m, ob.muon_hparams(lr=1.0, weight_decay=0.0, scale=ob.OB_MUON_PLAIN), work)
    for t in (0, 1, 2, 3, 200, 399, 401, 428, 429):
        u = grads[t].double()
        far = float((-params[t].double() - exact(u, 5, 1e-7 / (1 - 0.95 ** 2))).square().sum().sqrt())
        eps = torch.finfo(params[t].dtype).eps / 2
        assert far <= norm_bound(u, 5) + eps * math.sqrt(sum(s for s in shapes[t])), t


def test_groups_of_a_large_list():
    """A tensor whose matrices pass the workspace's limit: as each matrix alone.  The sums are the same bits in every tile, but a
    kernel may round fma(...) to fp16 once or by way of fp32 (a conversion fused into it or not), so the two X are two results
    within the bound of the exact one: twice the bound apart at most, times the update's factor, and each parameter half a step of
    bf16 more on both sides."""
    E, r, c = 70, 1024, 8192
    l, plan, grads, params, m, work = make([(E, r, c)], "bf16", "bf16", seed=2)
    assert plan.workspace_bytes < E * r * c * 4
    m0, p0 = m.clone(), params[0].clone()
    ob.ob_muon_step(plan, grads, params, m, ob.muon_hparams(lr=0.1), work)
    l1 = ob.ob_tensors_create([r * c], torch.bfloat16, torch.bfloat16)
    plan1 = ob.ob_muon_create(l1, [(r, c)])
    work1 = torch.empty(plan1.workspace_bytes, dtype=torch.uint8, device="cuda")
    for e in (0, 1, 33, 56, 57, 69):
        m1, p1 = m0.view(E, -1)[e].clone(), p0[e].clone()
        ob.ob_muon_step(plan1, [grads[0][e]], [p1], m1, ob.muon_hparams(lr=0.1), work1)
        assert torch.equal(m1, m.view(E, -1)[e])
        g, old = grads[0][e].double(), m0.view(E, r, c)[e].double()
        mu = float(torch.tensor(0.95))
        u = (1 - mu) * g + mu * (mu * old + (1 - mu) * g)
        far = (p1.double() - params[0][e].double()).square().sum().sqrt()
        size = torch.maximum(p1.double().abs(), params[0][e].double().abs()).square().sum().sqrt()
        assert float(far) <= 0.1 * 0.2 * math.sqrt(c) * 2 * norm_bound(u, 5) + 2 * 2.0 ** -8 * float(size)
        assert float((p1 != params[0][e]).double().mean()) < 0.5   # and no wholly other matrix


def test_class_graph_state_and_equal_bits():
    shapes = [(48, 32), (3, 24, 40), (130, 70)]
    gen = torch.Generator("cuda").manual_seed(0)
    start = [torch.randn(*s, generator=gen, device="cuda") * 0.02 for s in shapes]
    grads = [torch.randn(*s, generator=gen, device="cuda").bfloat16() for s in shapes]

    def new(**kw):
        return ob.Muon([torch.nn.Parameter(x.bfloat16()) for x in start], lr=0.02, master=True, max_norm=1.0, **kw)

    a, b = new(), new()
    for k in range(3):
        a.step([g * (k + 1) for g in grads])
    # captured and replayed, with eager work between
    static = [g.clone() for g in grads]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.step(static)
    for k in range(3):
        for x, y in zip(static, grads):
            x.copy_(y * (k + 1))
        g.replay()
        torch.cuda.synchronize()
    assert a.steps() == b.steps() == 3
    assert torch.equal(a.m, b.m) and torch.equal(a.master, b.master)
    assert all(torch.equal(x, y) for x, y in zip(a.params, b.params))
    c = new()
    c.load_state_dict(a.state_dict())
    for x, y in zip(c.params, a.params):
        x.data.copy_(y)
    for o in (a, c):
        o.set_lr_scale(0.5)
        o.step(grads)
    assert c.steps() == 4 and torch.equal(a.master, c.master) and all(torch.equal(x, y) for x, y in zip(a.params, c.params))
    # without a norm; a loss scale then is refused
    d = ob.Muon([torch.nn.Parameter(x.clone()) for x in start], lr=0.02)
    version = d.params[0]._version
    for p, x in zip(d.params, grads):
        p.grad = x.float()
    d.params[1].grad = None
    d.step()
    assert d.steps() == 1 and d.params[0]._version > version and torch.equal(d.params[1], start[1])
    with pytest.raises(ValueError, match="loss scale"):
        d.step(loss_scale=2.0)
    with pytest.raises(ValueError, match="m must"):
        d.load_state_dict({"step": 1, "m": torch.zeros(5)})


def test_two_captured_steps_with_their_own_workspaces():
    """Graphs of two plans replayed in turn and on two streams."""
    runs = []
    for seed in (1, 2):
        l, plan, grads, params, m, work = make([(64, 96), (40, 24)], seed=seed)
        hp = ob.muon_hparams(lr=0.1)
        want, m1 = [p.clone() for p in params], m.clone()
        other = torch.empty_like(work)
        for _ in range(4):
            ob.ob_muon_step(plan, grads, want, m1, hp, other)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ob.ob_muon_step(plan, grads, params, m, hp, work)
        runs.append((g, params, want, m, m1, plan, grads, work, hp))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        runs[0][0].replay()
        with torch.cuda.stream(side):
            runs[1][0].replay()
    torch.cuda.synchronize()
    for _, params, want, m, m1, *_ in runs:
        assert torch.equal(m, m1) and all(torch.equal(x, y) for x, y in zip(params, want))


def test_refusals():
    l, plan, grads, params, m, work = make([(8, 4)])
    hp = ob.muon_hparams()
    kept = params[0].clone()
    with pytest.raises(ValueError, match="no matrix"):
        ob.ob_muon_create(l, [(32,)])
    with pytest.raises(ValueError, match="elements"):
        ob.ob_muon_create(l, [(8, 5)])
    with pytest.raises(ValueError, match="entries"):
        ob.ob_muon_create(l, [(8, 4), (8, 4)])
    _, large, g2, p2, m2, work2 = make([(200, 300)])
    with pytest.raises(ValueError, match="bytes"):
        ob.ob_muon_step(large, g2, p2, m2, hp, work2[:-1])
    with pytest.raises(TypeError, match="workspace"):
        ob.ob_muon_step(large, g2, p2, m2, hp, None)
    with pytest.raises(TypeError, match="workspace"):
        ob.ob_muon_step(large, g2, p2, m2, hp, work2.view(torch.int8))
    with pytest.raises(TypeError, match="muon_hparams"):
        ob.ob_muon_step(plan, grads, params, m, ob.adamw_hparams(), work)
    with pytest.raises(ValueError, match="m must have"):
        ob.ob_muon_step(plan, grads, params, m[:8], hp, work)
    with pytest.raises(TypeError, match="grads"):
        ob.ob_muon_step(plan, [grads[0].half()], params, m, hp, work)
    with pytest.raises(TypeError, match="control"):
        ob.ob_muon_step(plan, grads, params, m, hp, work, norm=(1.0, 1.0))
    for bad in (dict(momentum=1.0), dict(eps=0.0), dict(lr=float("nan")), dict(iterations=17), dict(scale=9)):
        with pytest.raises(ob.ObError):
            ob.ob_muon_step(plan, grads, params, m, ob.muon_hparams(**bad), work)
    with pytest.raises(ValueError, match="no matrix"):
        ob.Muon([torch.zeros(8, device="cuda")])
    with pytest.raises(ValueError, match="scale"):
        ob.Muon([torch.zeros(8, 8, device="cuda")], scale="big")
    plan.destroy()
    with pytest.raises(ValueError, match="destroyed"):
        ob.ob_muon_step(plan, grads, params, m, hp, work)
    assert torch.equal(params[0], kept)
