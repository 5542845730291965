"""OneBitAdam and OneBitLamb with max_norm: a step whose gradient's norm is not finite changes nothing."""
import pytest
import torch

import adam_ob_compress_amd as ob

pytestmark = pytest.mark.gpu
STATES = ("err", "m", "v", "p", "words", "scales", "signs", "nonfinite", "err_sumsq", "plus_count", "ratios")


def make(cls, n, freeze_step, max_norm=0.5, err=torch.float32, **kw):
    plan = ob.ob_plan_create(n, chunk_size=1 << 14)
    gen = torch.Generator("cuda").manual_seed(n)
    state = [torch.randn(n, generator=gen, device="cuda") * 1e-2 for _ in range(4)]
    state[0] = state[0].to(err)
    state[2].square_()
    return cls(plan, *state, lr=1e-3, freeze_step=freeze_step, max_norm=max_norm, int8_signs=True, count_nonfinite=True,
               diagnostics=True, **kw)


def states(opt):
    return {k: getattr(opt, k).clone() for k in STATES if getattr(opt, k, None) is not None}


def gradient(n, dtype, seed, bad=None, at=0):
    g = torch.randn(n, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)
    if bad is not None:
        g[at] = bad
    return g


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("freeze_step", [0, 9])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("cls", [ob.OneBitAdam, ob.OneBitLamb])
def test_one_bad_element_leaves_the_step_out(cls, dtype, freeze_step, bad):
    n = 70_003
    for err in (torch.float32, torch.bfloat16, torch.float16):
        a, b = make(cls, n, freeze_step, err=err), make(cls, n, freeze_step, err=err)
        for k, at in enumerate((0, None, n - 1, 40_000, None)):
            before = states(a)
            kind = a.step(gradient(n, dtype, k, None if at is None else bad, at or 0))
            assert kind == ("dense" if freeze_step else "compressed")
            if at is None:
                assert bool(a.norm.isfinite())
                b.step(gradient(n, dtype, k))
            else:
                assert not bool(a.norm.isfinite())
                for name, x in states(a).items():
                    assert torch.equal(x, before[name]), (name, at)
        for name, x in states(a).items():   # as if those steps had never been
            assert torch.equal(x, getattr(b, name)) and (name in ("scales", "ratios") or bool(x.isfinite().all())), name
    assert a.step_index == 5


@pytest.mark.parametrize("freeze_step", [0, 9])
@pytest.mark.parametrize("cls", [ob.OneBitAdam, ob.OneBitLamb])
def test_replays_and_the_plans_other_steps(cls, freeze_step):
    """A captured step looks at the norm of each replay; the plan's other calls do not look at it."""
    n = 50_001
    a, b = make(cls, n, freeze_step), make(cls, n, freeze_step)
    g = gradient(n, torch.float32, 0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(g)
    for k, bad in enumerate((None, float("nan"), None, float("inf"), float("inf"), None)):
        before = states(a)
        g.copy_(gradient(n, torch.float32, k, bad, 77))
        graph.replay()
        torch.cuda.synchronize()
        if bad is None:
            b.step(gradient(n, torch.float32, k))
            assert all(torch.equal(x, getattr(b, name)) for name, x in states(a).items()), k
        else:
            assert all(torch.equal(x, before[name]) for name, x in states(a).items()), k
    # an ordinary step with the same plan, after one that was left out
    a.step(gradient(n, torch.float32, 1, float("nan")))
    p = a.p.clone()
    ob.ob_adam_warmup_step(a.plan, gradient(n, torch.float32, 2), a.m, a.v, a.p, ob.hparams(lr=1e-3))
    assert not torch.equal(a.p, p) and bool(a.p.isfinite().all())


def test_large_chunks_and_groups(monkeypatch):
    """Chunks whose partial sums a launch of their own adds, and passes over several groups."""
    n = 5_000_001
    for env, chunk in (({"OB_BLOCK_ELEMS": "1024"}, n), ({"OB_GROUP_BYTES": str(1 << 20)}, 1 << 16)):
        for k, v in env.items():
            monkeypatch.setenv(k, v)
        plan = ob.ob_plan_create(n, chunk_size=chunk)
        state = [torch.zeros(n, device="cuda") for _ in range(4)]
        opt = ob.OneBitAdam(plan, *state, lr=1e-3, max_norm=1.0)
        opt.step(gradient(n, torch.float32, 1))
        before = [x.clone() for x in (*state, opt.words, opt.scales)]
        opt.step(gradient(n, torch.float32, 2, float("inf"), n - 1))
        assert all(torch.equal(x, y) for x, y in zip(before, (*state, opt.words, opt.scales)))
        opt.step(gradient(n, torch.float32, 3))
        assert not torch.equal(opt.p, before[3]) and bool(opt.p.isfinite().all())
        for k in env:
            monkeypatch.delenv(k)
