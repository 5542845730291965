"""The Muon step on matrices beyond a compute unit's LDS: the launches that large matrices take, in all that a call can ask for.

Tolerances: those of test_gpu_muon.py, whose bounds are used here.
"""
import math

import pytest
import torch

import adam_ob_compress_amd as ob
from test_gpu_muon import DT, U, directions, element_bound, exact, make, norm_bound, part

pytestmark = pytest.mark.gpu

# Lists by the tiles that their plans take for the Gram matrix, the polynomial and the step; sides that are no multiples of 8 or of
# a tile, both orientations in one launch.  tests/test_muon_limits.py holds that these are the tiles.
LISTS = {"64-64-64": [(2, 203, 300), (300, 203), (169, 178), (171, 169)],
         "64-64-128": [(7, 521, 777), (6, 777, 520)],
         "64-64-256": [(100, 201, 203), (103, 202, 197)],
         "128-128-256": [(4, 1100, 1301), (4, 1303, 1101)],
         "256-256-256": [(32, 509, 1403), (1403, 510), (31, 1402, 507)]}


def some(E):
    """A few of a tensor's matrices, its first and last among them."""
    return sorted({0, E // 3, E - 1})


@pytest.mark.parametrize("iterations", [1, 2])
@pytest.mark.parametrize("shapes", LISTS.values(), ids=LISTS)
def test_each_element(shapes, iterations):
    """Every element of X, of tall and wide matrices with ragged ends, by every tile."""
    l, plan, grads, params, m, work = make(shapes, seed=len(shapes))
    assert plan.workspace_bytes > 0
    mu = float(torch.tensor(0.9))
    want = directions(l, shapes, grads, m, mu, True)
    for p in params:
        p.zero_()
    work.fill_(255)   # of any content: NaN in fp16
    hp = ob.muon_hparams(lr=1.0, momentum=mu, weight_decay=0.0, iterations=iterations, scale=ob.OB_MUON_PLAIN)
    ob.ob_muon_step(plan, grads, params, m, hp, work)
    for t, (s, (new, u), p) in enumerate(zip(shapes, want, params)):
        assert ((part(l, m, t, s).double() - new).abs() <= 4 * U * new.abs() + 1e-12).all()
        y, x = p.view(-1, *s[-2:]), u.view(-1, *s[-2:])
        for e in some(len(y)):
            far = (-y[e].double() - exact(x[e], iterations)).abs()
            bound = element_bound(x[e], iterations)
            assert (far <= bound + 4 * U).all(), (t, e, float((far / bound).max()))


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("shapes", LISTS.values(), ids=LISTS)
def test_five_iterations(shapes, nesterov):
    l, plan, grads, params, m, work = make(shapes, seed=7, kind="graded")
    want = directions(l, shapes, grads, m, float(torch.tensor(0.95)), nesterov)
    for p in params:
        p.zero_()
    ob.ob_muon_step(plan, grads, params, m, ob.muon_hparams(lr=1.0, momentum=0.95, weight_decay=0.0, scale=ob.OB_MUON_PLAIN,
                                                            nesterov=nesterov), work)
    for s, (_, u), p in zip(shapes, want, params):
        y, x = p.view(-1, *s[-2:]), u.view(-1, *s[-2:])
        for e in some(len(y)):
            far = float((-y[e].double() - exact(x[e], 5)).square().sum().sqrt())
            assert far <= norm_bound(x[e], 5), (s, e)


SCALES = {ob.OB_MUON_PLAIN: lambda R, K: 1.0, ob.OB_MUON_SHAPE: lambda R, K: math.sqrt(max(1.0, R / K)),
          ob.OB_MUON_MATCH_RMS: lambda R, K: 0.2 * math.sqrt(max(R, K))}


@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("g,p", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("shapes", LISTS.values(), ids=LISTS)
def test_parameters(shapes, g, p, master):
    """Types, masters, decay, rates and scales: the parameters' line from the X that the same step gives on zero parameters in fp32.
    Parameters and gradients start at any element."""
    T = len(shapes)
    mults = [(1.0, 0.5, 2.0, 1.0)[:T], (0.0, 1.0, 3.0, 1.0)[:T]]
    sizes = [math.prod(s) for s in shapes]
    l0, plan, grads, x, m, work = make(shapes, g, "f32", seed=3)
    start_m = m.clone()
    for q in x:
        q.zero_()
    ob.ob_muon_step(plan, grads, x, m, ob.muon_hparams(lr=1.0, weight_decay=0.0, scale=ob.OB_MUON_PLAIN), work)
    l = ob.ob_tensors_create(sizes, DT[g], DT[p], *mults)
    plan = ob.ob_muon_create(l, shapes)
    gen = torch.Generator("cuda").manual_seed(5)
    old = [torch.randn(*s, generator=gen, device="cuda") * 0.02 for s in shapes]
    odd = [torch.cat([q.new_zeros(3), q.flatten(), q.new_zeros(1)])[3:-1].view(q.shape) for q in grads]
    assert all(q.data_ptr() % 16 for q in odd)
    lr, wd = float(torch.tensor(0.01)), float(torch.tensor(0.1))
    for scale in SCALES:
        around = [torch.full((n + 2,), 7.0, dtype=DT[p], device="cuda") for n in sizes]
        params = [q[1:-1].view(s) for q, s in zip(around, shapes)]
        flat = torch.zeros(l.state_elems, device="cuda") if master else None
        for t, (q, o) in enumerate(zip(params, old)):
            q.copy_(o)
            if master:
                part(l, flat, t, o.shape).copy_(o)
        m2 = start_m.clone()
        ob.ob_muon_step(plan, odd, params, m2, ob.muon_hparams(lr=lr, weight_decay=wd, scale=scale), work, master=flat)
        assert torch.equal(m, m2)
        for t, (s, y, o) in enumerate(zip(shapes, x, old)):
            f = SCALES[scale](*s[-2:])
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
            assert float(around[t][0]) == float(around[t][-1]) == 7.0   # what lies beside the parameters


@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("shapes", [LISTS["64-64-64"], LISTS["128-128-256"], LISTS["256-256-256"]], ids=["64", "128", "256"])
def test_control_block(shapes, master):
    """Clipping, the rate's factor and steps left out, with bf16 parameters."""
    l, plan, grads, params, m, work = make(shapes, "f32", "bf16")
    start, m0 = [p.clone() for p in params], m.clone()
    flat = torch.randn(l.state_elems, device="cuda") * 0.02 if master else None
    flat0 = flat.clone() if master else None
    ctl = ob.control_create()
    f = ob.control_fields(ctl)
    f["lr_scale"].fill_(0.5)
    ob.ob_muon_step(plan, grads, params, m, ob.muon_hparams(lr=0.02), work, flat, ctl, norm=(0.25, 1e-3))
    total = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    assert abs(float(f["norm"]) - 0.25 * total) <= 1.01 * U * total and int(f["step"]) == 1
    # the same step with the gradients scaled by hand and half the rate
    again, m1 = [p.clone() for p in start], m0.clone()
    ob.ob_muon_step(plan, [g * f["grad_scale"] for g in grads], again, m1, ob.muon_hparams(lr=0.01), work, flat0)
    assert torch.equal(m, m1) and all(torch.equal(x, y) for x, y in zip(params, again))
    assert not master or torch.equal(flat, flat0)
    assert not any(torch.equal(x, y) for x, y in zip(params, start))
    # a norm that is not finite: nothing changes
    grads[-1].view(-1)[17] = float("nan")
    ob.ob_muon_step(plan, grads, params, m, ob.muon_hparams(lr=0.02), work, flat, ctl, norm=(1.0, 0.0))
    assert torch.equal(m, m1) and all(torch.equal(x, y) for x, y in zip(params, again))
    assert not master or torch.equal(flat, flat0)
    assert int(f["step"]) == 1 and int(f["skipped"]) == 1


@pytest.mark.parametrize("shapes", [LISTS["64-64-64"] + [(40, 24)], LISTS["64-64-256"], LISTS["256-256-256"]], ids=["64", "64-256", "256"])
def test_missing_gradients_zeros_and_bad_values(shapes):
    """One group's tensors with and without a gradient, a matrix of zeros, a NaN and an infinity in one matrix of many."""
    l, plan, grads, params, m, work = make(shapes, "bf16", "f32")
    work.fill_(255)
    kept, m0 = [p.clone() for p in params], m.clone()
    hp = ob.muon_hparams(lr=0.1)
    want, m1 = [p.clone() for p in params], m.clone()
    ob.ob_muon_step(plan, grads, want, m1, hp, work)
    work.fill_(255)
    given = [g if j != 1 else None for j, g in enumerate(grads)]
    ob.ob_muon_step(plan, given, params, m, hp, work)
    for j, s in enumerate(shapes):
        assert torch.equal(params[j], kept[j] if j == 1 else want[j]) and params[j].isfinite().all()
        assert torch.equal(part(l, m, j, s), part(l, m0 if j == 1 else m1, j, s))
    ob.ob_muon_step(plan, [None] * len(shapes), params, m, hp, work)
    assert torch.equal(params[0], want[0])
    # in the first tensor's last matrix: zeros, whose step is the decay, then a NaN, then an infinity; the other matrices are as they were
    for bad in (None, float("nan"), float("inf")):
        again, m2 = [p.clone() for p in kept], m0.clone()
        x, y = grads[0].view(-1, *shapes[0][-2:])[-1], part(l, m2, 0, shapes[0]).view(-1, *shapes[0][-2:])[-1]
        if bad is None:
            x.zero_()
            y.zero_()
        else:
            x[3, 5] = bad
        work.fill_(255)
        ob.ob_muon_step(plan, grads, again, m2, ob.muon_hparams(lr=0.1, weight_decay=0.5), work)
        new, old = again[0].view(-1, *shapes[0][-2:])[-1], kept[0].view(-1, *shapes[0][-2:])[-1]
        if bad is None:
            decay = torch.tensor(0.5, device="cuda")
            assert torch.equal(new, torch.addcmul(old, old, decay, value=-float(torch.tensor(0.1))))
        else:
            assert not new.isfinite().any()
        assert all(p.isfinite().all() for p in again[1:])
        assert again[0].view(-1, *shapes[0][-2:])[:-1].isfinite().all()


def test_mixed_types_and_many_tensors():
    """Types in turn, more tensors than a launch takes, large matrices and small ones, at any element."""
    T = 430
    shapes = [((169, 200), (24, 8), (203, 177))[j % 3] for j in range(T)]
    types = [("f32", "bf16")[j % 2] for j in range(T)]
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
    assert plan.workspace_bytes > 0
    m = torch.zeros(l.state_elems, device="cuda")
    work = torch.full((plan.workspace_bytes,), 255, dtype=torch.uint8, device="cuda")
    ob.ob_muon_step(plan, grads, params, m, ob.muon_hparams(lr=1.0, weight_decay=0.0, scale=ob.OB_MUON_PLAIN), work)
    for t in (0, 1, 2, 3, 200, 399, 401, 402, 428, 429):
        u = grads[t].double()
        x = exact(u, 5, 1e-7 / (1 - 0.95 ** 2))
        far = float((-params[t].double() - x).square().sum().sqrt())
        eps = torch.finfo(params[t].dtype).eps / 2
        bound = norm_bound(u, 5)
        assert far <= bound + eps * (float(x.square().sum().sqrt()) + bound), t


def test_two_captured_steps_with_their_own_workspaces():
    """Graphs of two plans replayed on two streams, with eager steps of others between; every replay against an eager step."""
    runs = []
    for seed, shapes in ((1, LISTS["64-64-64"]), (2, LISTS["256-256-256"])):
        l, plan, grads, params, m, work = make(shapes, "bf16", "bf16", seed=seed)
        assert plan.workspace_bytes > 0
        hp = ob.muon_hparams(lr=0.1)
        want, m1, other = [p.clone() for p in params], m.clone(), torch.empty_like(work)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ob.ob_muon_step(plan, grads, params, m, hp, work)
        runs.append((g, params, want, m, m1, plan, grads, other, hp, work))
    side = torch.cuda.Stream()
    for k in range(4):
        side.wait_stream(torch.cuda.current_stream())
        runs[0][0].replay()
        with torch.cuda.stream(side):
            runs[1][0].replay()
        torch.cuda.current_stream().wait_stream(side)
        for _, params, want, m, m1, plan, grads, other, hp, _ in runs:
            ob.ob_muon_step(plan, grads, want, m1, hp, other)
            torch.cuda.synchronize()
            assert torch.equal(m, m1) and all(torch.equal(x, y) for x, y in zip(params, want)), k


def test_class_with_groups_and_state():
    shapes = [(300, 203), (3, 200, 264), (40, 24), (520, 700)]
    gen = torch.Generator("cuda").manual_seed(0)
    start = [torch.randn(*s, generator=gen, device="cuda") * 0.02 for s in shapes]
    grads = [torch.randn(*s, generator=gen, device="cuda").bfloat16() for s in shapes]

    def new():
        ps = [torch.nn.Parameter(x.bfloat16()) for x in start]
        o = ob.Muon([{"params": ps[:2]}, {"params": ps[2:], "lr": 0.04, "weight_decay": 0.0}], lr=0.02, master=True, max_norm=1.0)
        for t, x in enumerate(start):
            part(o.list, o.master, t, x.shape).copy_(x)
        return o

    a, b = new(), new()
    assert a.plan.workspace_bytes > 0
    static = [g.clone() for g in grads]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step(static)
    for k in range(3):
        a.step([g * (k + 1) for g in grads])
        for x, y in zip(static, grads):
            x.copy_(y * (k + 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.m, b.m) and torch.equal(a.master, b.master)
        assert all(torch.equal(x, y) for x, y in zip(a.params, b.params)), k
    c = new()
    c.load_state_dict(a.state_dict())
    for x, y in zip(c.params, a.params):
        x.data.copy_(y)
    for o in (a, c):
        o.set_lr_scale(0.5)
        o.step(grads)
    assert c.steps() == a.steps() == 4 and torch.equal(a.master, c.master)
    assert all(torch.equal(x, y) for x, y in zip(a.params, c.params))


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
    part_of = (torch.randn(side, at.numel(), generator=gen, device="cuda") * torch.linspace(0.2, 2, side, device="cuda")[:, None]).bfloat16()
    g = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    (g.t() if rows > cols else g)[:, at] = part_of
    p = torch.zeros_like(g)
    l = ob.ob_tensors_create([g.numel()], torch.bfloat16, torch.bfloat16)
    plan = ob.ob_muon_create(l, [g.shape])
    m = torch.zeros(l.state_elems, device="cuda")
    work = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    ob.ob_muon_step(plan, [g], [p], m, ob.muon_hparams(lr=1.0, momentum=0.0, weight_decay=0.0, iterations=iterations,
                                                      scale=ob.OB_MUON_PLAIN), work)
    p = p.t() if rows > cols else p
    got, want, bound = p[:, at].double(), exact(part_of, iterations), element_bound(part_of, iterations)
    assert ((got + want).abs() <= bound + (2.0 ** -8 + 4 * U) * (want.abs() + bound)).all()
    p[:, at] = 0
    assert not p.any()   # nothing but the decay, which is 0, where there is no gradient


def test_longer_matrices_are_refused():
    for shape in ((64, 17_100_000), (17_100_000, 64), (8, 160_000_000)):
        l = ob.ob_tensors_create([math.prod(shape)], torch.bfloat16, torch.bfloat16)
        with pytest.raises(ob.ObError):
            ob.ob_muon_create(l, [shape])
