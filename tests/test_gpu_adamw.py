"""The steps over lists of tensors on the GPU against plain references in 64 bits (tests/_adamw_ref.py).

Tolerances, with eps the distance of 1 from the next fp32 number (2^-23):
  * fp32 states: a line is evaluated in double and rounded once, so it is off by at most half a step,
    eps/2 |x|, of its fp64 value; the double evaluation itself adds below 2^-48 of the terms' magnitudes.
  * 8-bit states: codes and scales are equal (every rounding is stated by the format).  The parameters' line in
    fp32: two roots and a reciprocal good to an ulp, six roundings: the update is off by less than 2^-20 of
    |m^/den| and the decay by 2^-22 of |wd p|, then half a step of the result.
  * 16-bit parameters: the rounding of one of the fp32 numbers that these tolerances allow.
  * the norm: fp64 sums, rounded to fp32 once: half a step.
"""
import ctypes

import numpy as np
import pytest
import torch

import _adamw_ref as ref
import adam_ob_compress_amd as ob
import oracle

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HP = dict(lr=3e-3, beta1=0.9, beta2=0.98, eps=1e-8, weight_decay=0.1)
EPS32 = 2.0 ** -23

SIZES = [1, 2, 3, 4, 5, 63, 64, 65, 0, 255, 256, 257, 1023, 1024, 1025, 4095, 4096, 4097, 9001]


@pytest.fixture(autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible MI355X"
    ob.lib()
    yield
    torch.cuda.synchronize()


def f64(t):
    return t.detach().cpu().double().numpy()


class Lists:
    """A list on the GPU: tensors at odd places between guard elements, states with guarded gaps."""

    def __init__(self, sizes, g, p, seed=0, master=False, bits=32, lr_mults=None, wd_mults=None, shift=True,
                 grad_sigma=1e-3):
        self.rng = np.random.default_rng(seed)
        T = len(sizes)
        self.sizes, self.bits, self.master_on = sizes, bits, master
        self.g = [g] * T if isinstance(g, str) else g
        self.p = [p] * T if isinstance(p, str) else p
        self.lr_mults, self.wd_mults = lr_mults or [1.0] * T, wd_mults or [1.0] * T
        self.list = ob.ob_tensors_create(sizes, [DT[x] for x in self.g], [DT[x] for x in self.p], lr_mults, wd_mults, DEV)
        N = self.N = self.list.state_elems
        self.off = [self.list.state_offset(t) for t in range(T)]
        self.inside = np.zeros(N, bool)
        for o, n in zip(self.off, sizes):
            self.inside[o:o + n] = True
        self.grad_sigma = grad_sigma
        self.shift = shift
        self.guards = []
        self.params = [self._place(self.rng.standard_normal(n) * 0.05, DT[d]) for n, d in zip(sizes, self.p)]
        self.draw_grads()
        m = self.rng.standard_normal(N) * 1e-3
        v = (self.rng.standard_normal(N) * 1e-3) ** 2
        m[~self.inside] = v[~self.inside] = 0
        self.m0, self.v0 = m.astype(np.float32), v.astype(np.float32)
        if bits == 32:
            self.m, self.v = self._state(self.m0, 7.0), self._state(self.v0, 7.0)
        else:
            mc, mq = ref.encode(self.m0, False)
            vc, vq = ref.encode(self.v0, True)
            self.mc, self.vc = self._state(mc, 77), self._state(vc, 77)
            self.mq, self.vq = torch.from_numpy(mq).to(DEV), torch.from_numpy(vq).to(DEV)
        self.master = None
        if master:
            # fp32 values near the 16-bit parameters; fp32 tensors' part is a guard
            w = np.full(N, 7.0, np.float32)
            for t, (o, n) in enumerate(zip(self.off, sizes)):
                if self.p[t] != "f32":
                    w[o:o + n] = f64(self.params[t]) * (1 + 1e-3 * self.rng.standard_normal(n))
            self.master = torch.from_numpy(w).to(DEV)

    def _place(self, x, dtype):
        n = len(x)
        a = int(self.rng.integers(1, 9)) if self.shift else 8
        buf = torch.full((n + 16,), 3.0, dtype=dtype, device=DEV)
        view = buf[a:a + n]
        view.copy_(torch.from_numpy(np.asarray(x)).to(DEV))
        self.guards.append((buf, a, n))
        return view

    def _state(self, x, gap):
        x = x.copy()
        x[~self.inside] = gap
        return torch.from_numpy(x).to(DEV)

    def draw_grads(self, none=()):
        self.grads = [None if t in none else self._place(self.rng.standard_normal(n) * self.grad_sigma, DT[d])
                      for t, (n, d) in enumerate(zip(self.sizes, self.g))]

    def snapshot(self):
        s = {"p": [f64(x) for x in self.params]}
        if self.bits == 32:
            s["m"], s["v"] = f64(self.m), f64(self.v)
        else:
            for k in ("mc", "mq", "vc", "vq"):
                s[k] = getattr(self, k).cpu().numpy().copy()
            mc, vc = s["mc"].copy(), s["vc"].copy()
            mc[~self.inside], vc[~self.inside] = 0, 0
            s["m"], s["v"] = ref.decode(mc, s["mq"], False), ref.decode(vc, s["vq"], True)
        if self.master is not None:
            s["master"] = f64(self.master)
        return s

    def step(self, hp, control=None, stream=None):
        if self.bits == 32:
            ob.ob_adamw_step(self.list, self.grads, self.params, self.m, self.v, hp, self.master, control, stream)
        else:
            ob.ob_adamw8_step(self.list, self.grads, self.params, self.mc, self.mq, self.vc, self.vq, hp, self.master,
                              control, stream)

    def check_guards(self):
        for buf, a, n in self.guards:
            x = buf.cpu().float()
            assert torch.all(x[:a] == 3.0) and torch.all(x[a + n:] == 3.0), "written beside a tensor"
        gaps = {"m": 7, "v": 7} if self.bits == 32 else {"mc": 77, "vc": 77}
        for k, value in gaps.items():
            assert np.all(getattr(self, k).cpu().numpy()[~self.inside] == value), f"gap of {k} written"
        if self.master is not None:
            keep = ~self.inside
            for t, (o, n) in enumerate(zip(self.off, self.sizes)):
                if self.p[t] == "f32":
                    keep[o:o + n] = True
            assert np.all(self.master.cpu().numpy()[keep] == 7.0), "the master's unused part written"

    def parts(self):
        """(tensor, state offset, elements, slice in the tensor) of what is compared: all of a tensor, or, as state blocks
        do not depend on each other, the first, last and some other blocks of a long one."""
        for j, (o, n) in enumerate(zip(self.off, self.sizes)):
            if 0 < n <= 1 << 20:
                yield j, o, n, slice(0, n)
            elif n:
                starts = [0, n // 256 * 256 - 8192] + [int(x) * 256 for x in self.rng.integers(32, n // 256 - 64, 12)]
                for a in starts:
                    b = min(n, a + (9000 if a == starts[1] else 2048))
                    yield j, o + a, b - a, slice(a, b)

    def check(self, before, hp, *, t, scale=1.0, lr_scale=1.0, bc=None, none=()):
        """The step from `before` against the reference."""
        after = self.snapshot()
        self.check_guards()
        b1, b2 = (1.0, 1.0) if not hp.bias_correction else bc or (ref.bc(hp.beta1, t), ref.bc(hp.beta2, t))
        sr = hp.rounding == ob.OB_ROUND_STOCHASTIC
        words = ref.philox_words(hp.sr_seed, t, self.N) if sr else None
        for j, o, n, part in self.parts():
            s, what = slice(o, o + n), f"tensor {j} ({n}, g {self.g[j]}, p {self.p[j]})"
            if j in none:
                assert np.array_equal(after["p"][j][part], before["p"][j][part]), what
                for k in ("m", "v") + (("master",) if self.master is not None else ()):
                    assert np.array_equal(after[k][s], before[k][s]), (what, k)
                continue
            g = f64(self.grads[j][part])
            use_master = self.master is not None and self.p[j] != "f32"
            p0 = before["master"][s] if use_master else before["p"][j][part]
            lr, wd = float(hp.lr) * lr_scale * float(np.float32(self.lr_mults[j])), float(hp.weight_decay) * float(np.float32(self.wd_mults[j]))
            kw = dict(lr=lr, beta1=hp.beta1, beta2=hp.beta2, eps=hp.eps, wd=wd, bc1=b1, bc2=b2, scale=scale)
            if self.bits == 32:
                m, v, p, u = ref.adamw(g, before["m"][s], before["v"][s], p0, **kw)
                for k, x in (("m", m), ("v", v)):
                    close(after[k][s], x, EPS32 / 2 * np.abs(x) * (1 + 1e-6) + 2.0 ** -149, (what, k))
                slack = 2.0 ** -46 * (np.abs(p0) + np.abs(lr * u))
            else:
                m, v = ref.adamw8_moments(g, before["m"][s], before["v"][s], beta1=hp.beta1, beta2=hp.beta2, scale=scale)
                for k, x, second in (("m", m, False), ("v", v, True)):
                    c, q = ref.encode(x, second, None if words is None else words[s])
                    assert np.array_equal(after[k + "q"][o // 256: o // 256 + len(q)], q, equal_nan=True), (what, k)
                    assert np.array_equal(after[k + "c"][s], c), (what, k, np.nonzero(after[k + "c"][s] != c)[0][:5])
                u = (m / b1) / (np.sqrt(v / b2) + float(np.float32(hp.eps)))
                p = p0 - lr * (u + wd * p0)
                slack = np.abs(lr) * (2.0 ** -20 * np.abs(u) + 2.0 ** -22 * np.abs(wd * p0))
            tol = EPS32 / 2 * np.abs(p) + slack * (1 + 1e-6) + 2.0 ** -149
            if use_master or self.p[j] == "f32":
                close(after["master"][s] if use_master else after["p"][j][part], p, tol, (what, "p"))
            if self.p[j] == "f32":
                continue
            if use_master:   # the copy is the rounding of the master that is there
                want = torch.from_numpy(after["master"][s]).float().to(DT[self.p[j]]).double().numpy()
                assert np.array_equal(after["p"][j][part], want), what
            else:
                lo, hi = (p - tol).astype(np.float32), (p + tol).astype(np.float32)
                if sr:   # up where the random bits are below the fraction: monotone in the value
                    pw = [from16(oracle.to_format_sr(x, self.p[j], hp.sr_seed, t | ref.PAR_STREAM, o), self.p[j]) for x in (lo, hi)]
                else:
                    pw = [torch.from_numpy(x).to(DT[self.p[j]]).double().numpy() for x in (lo, hi)]
                assert np.all((after["p"][j][part] >= np.minimum(*pw)) & (after["p"][j][part] <= np.maximum(*pw))), what
        return after


def from16(bits, fmt):
    return oracle.from_format(bits, fmt).astype(np.float64)


def close(got, want, tol, what):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:3], want[bad][:3], tol[bad][:3] if np.ndim(tol) else tol)


def hparams(**kw):
    return ob.adamw_hparams(**{**HP, **kw})


# ---- the steps ----

@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("g,p,master", [("f32", "f32", False), ("bf16", "f32", False), ("f16", "f32", False),
                                        ("bf16", "bf16", False), ("f16", "f16", False), ("f32", "bf16", False),
                                        ("bf16", "bf16", True), ("f16", "f16", True), ("f32", "bf16", True),
                                        ("f32", "f16", True)])
@pytest.mark.parametrize("stochastic", [False, True])
def test_step(bits, g, p, master, stochastic):
    """Every size around the kernels' borders, tensors at odd addresses, three steps with new gradients."""
    L = Lists(SIZES, g, p, seed=bits, master=master, bits=bits, lr_mults=[1.0, 0.5, 2.0] * 6 + [1.0],
              wd_mults=[0.0, 1.0] * 9 + [3.0])
    for t in (1, 2, 1000):
        hp = hparams(step=t, rounding=int(stochastic), sr_seed=0xABCDEF0123456789)
        before = L.snapshot()
        L.step(hp)
        torch.cuda.synchronize()
        L.check(before, hp, t=t)
        L.draw_grads()


@pytest.mark.parametrize("g,p,master", [("bf16", "f32", False), ("bf16", "bf16", False), ("f32", "f16", False),
                                        ("f16", "bf16", True)])
@pytest.mark.parametrize("stochastic", [False, True])
def test_long_tensors(g, p, master, stochastic):
    """More than 2048 work blocks in a launch, where a wave takes four state blocks: whole and ragged spans."""
    L = Lists([9_000_000, 300, 8_500_003, 1025], g, p, seed=15, master=master, bits=8)
    hp = hparams(step=9, rounding=int(stochastic), sr_seed=3)
    before = L.snapshot()
    L.step(hp)
    torch.cuda.synchronize()
    L.check(before, hp, t=9)


@pytest.mark.parametrize("bits", [32, 8])
def test_aligned_whole_blocks_without_bias_correction(bits):
    L = Lists([1024, 4096, 8192, 256], "f32", "f32", seed=5, bits=bits, shift=False)
    hp = hparams(bias_correction=False, step=0, weight_decay=0.0)
    before = L.snapshot()
    L.step(hp)
    torch.cuda.synchronize()
    L.check(before, hp, t=0)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("master", [False, True])
def test_many_tensors_of_mixed_types(bits, master):
    """More tensors than one launch's arguments hold, of every pair of types, some without a gradient."""
    rng = np.random.default_rng(8)
    T = 1100
    sizes = [int(x) for x in rng.integers(0, 600, T)]
    kinds = ["f32", "bf16", "f16"]
    L = Lists(sizes, [kinds[i] for i in rng.integers(0, 3, T)], [kinds[i] for i in rng.integers(0, 3, T)], seed=9,
              bits=bits, master=master)
    none = set(int(i) for i in rng.integers(0, T, 100))
    L.draw_grads(none)
    hp = hparams(step=7)
    before = L.snapshot()
    L.step(hp)
    torch.cuda.synchronize()
    L.check(before, hp, t=7, none=none)


def test_one_type_in_several_launches():
    L = Lists([300 + i for i in range(700)], "bf16", "f32", seed=10, bits=8)
    hp = hparams(step=3)
    before = L.snapshot()
    L.step(hp)
    torch.cuda.synchronize()
    L.check(before, hp, t=3)


@pytest.mark.parametrize("g", ["f32", "bf16"])
@pytest.mark.parametrize("bias_correction", [False, True])
def test_fp32_step_is_the_dense_step(g, bias_correction):
    """Without decay the bits of ob_adam_warmup_step."""
    n = 300_001
    rng = np.random.default_rng(2)
    m, v, p = (torch.from_numpy((rng.standard_normal(n) * 1e-2).astype(np.float32)).to(DEV) for _ in range(3))
    v.square_()
    gr = torch.from_numpy(rng.standard_normal(n) * 1e-2).to(DEV).to(DT[g])
    m2, v2, p2 = torch.zeros((n + 255) // 256 * 256, device=DEV), torch.zeros((n + 255) // 256 * 256, device=DEV), p.clone()
    m2[:n], v2[:n] = m, v
    plan = ob.ob_plan_create(n, chunk_size=1 << 16)
    lst = ob.ob_tensors_create([n], DT[g], torch.float32)
    for t in (1, 2, 3):
        ob.ob_adam_warmup_step(plan, gr, m, v, p, ob.hparams(lr=1e-3, bias_correction=bias_correction, step=t))
        ob.ob_adamw_step(lst, [gr], [p2], m2, v2, ob.adamw_hparams(lr=1e-3, weight_decay=0.0, step=t, bias_correction=bias_correction))
    assert torch.equal(p, p2) and torch.equal(m, m2[:n]) and torch.equal(v, v2[:n])


@pytest.mark.parametrize("bits", [32, 8])
def test_special_values(bits):
    """NaN and infinite gradients, zero gradients with zero moments, tiny and huge gradients."""
    L = Lists([256, 256, 256, 256, 256, 256, 3], "f32", "f32", seed=3, bits=bits, shift=False)
    L.grads[0][7] = float("nan")
    L.grads[1][9] = float("inf")
    L.grads[2].mul_(1e-25)
    L.grads[3].mul_(1e18)
    L.grads[4].zero_()
    if bits == 32:
        for x in (L.m, L.v):
            x[2 * 256:5 * 256] = 0
    else:
        for x in (L.mq, L.vq):
            x[2:5] = 0
    hp = hparams(step=5)
    before = L.snapshot()
    L.step(hp)
    torch.cuda.synchronize()
    after = L.snapshot()
    p = after["p"]
    if bits == 32:
        assert np.isnan(p[0][7]) and np.isfinite(np.delete(p[0], 7)).all()
        assert np.isnan(after["m"][7]) and np.isinf(after["m"][256 + 9])
    else:
        # the block reads as NaN from here on; its other parameters took this step's finite values
        assert np.isnan(p[0][7]) and np.isfinite(np.delete(p[0], 7)).all()
        assert np.isnan(after["mq"][0]) and np.isnan(after["vq"][1]) and not after["mc"][:512].any()
        assert np.isnan(after["m"][:512]).all()
        # 1e-28 squared is below 2^-96: v is held as zeros; m is not
        assert after["vq"][2] == 0 and after["mq"][2] > 0
    # no gradient and no moments: decay only
    x = before["p"][4]
    close(p[4], x - float(hp.lr) * float(hp.weight_decay) * x, EPS32 * np.abs(x), "decay")
    for j in (2, 3, 5, 6):
        assert np.isfinite(p[j]).all(), j
    L.check_guards()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("stochastic", [False, True])
def test_parameters_that_nothing_moves_keep_their_bits(bits, p, stochastic):
    """No gradient, moments or decay: zeros, subnormal numbers and the largest ones come back as they were."""
    L = Lists([300], p, p, seed=8, bits=bits)
    top = torch.finfo(DT[p]).max
    tiny = torch.finfo(DT[p]).smallest_normal
    L.params[0][:8] = torch.tensor([0.0, -0.0, tiny, tiny / 4, -tiny / 4, top, -top, 1.0], device=DEV).to(DT[p])
    L.grads[0].zero_()
    for x in ((L.m, L.v) if bits == 32 else (L.mq, L.vq)):
        x[:300 if bits == 32 else 2] = 0
    want = L.params[0].clone()
    hp = hparams(weight_decay=0.0, step=1, rounding=int(stochastic), sr_seed=4)
    L.step(hp)
    torch.cuda.synchronize()
    assert torch.equal(L.params[0].view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("p", ["bf16", "f16"])
@pytest.mark.parametrize("bits", [32, 8])
def test_copies_of_extreme_masters(p, bits):
    """Masters that are subnormal in the copy's type, at its largest value and beyond it, and NaN."""
    L = Lists([256, 7], "f32", p, seed=8, bits=bits, master=True)
    fi = torch.finfo(DT[p])
    x = torch.linspace(-3, 3, 256, device=DEV) * fi.smallest_normal
    x[:7] = torch.tensor([float("nan"), float("inf"), fi.max, -fi.max * (1 - fi.eps / 8), min(fi.max * (1.0 + fi.eps / 2), 3.4e38),
                          fi.tiny / 2 ** 9, 1.0], device=DEV)
    L.master[:256] = x
    for g in L.grads:
        g.zero_()
    for y in ((L.m, L.v) if bits == 32 else (L.mq, L.vq)):
        y[:] = 0
    L.step(hparams(weight_decay=0.0, step=1))
    torch.cuda.synchronize()
    # the infinite one turns NaN: the line's decay is 0 * inf
    assert torch.equal(L.master[:256].view(torch.int32)[2:], x.view(torch.int32)[2:]) and torch.isnan(L.master[:2]).all()
    got, want = L.params[0].cpu(), x.cpu().to(DT[p])
    assert torch.isnan(got[:2]).all() and torch.equal(got[2:].view(torch.int16), want[2:].view(torch.int16))


def test_huge_tensor():
    """Offsets past 2^32 elements: one bf16 tensor with 8-bit states; the places around 2^31, 2^32 and the end."""
    n = (1 << 32) + 4099
    lst = ob.ob_tensors_create([5, n], torch.bfloat16, torch.bfloat16)
    N, o = lst.state_elems, lst.state_offset(1)
    g = torch.full((n,), 1e-3, dtype=torch.bfloat16, device=DEV)
    p = torch.full((n,), 0.5, dtype=torch.bfloat16, device=DEV)
    small = [torch.ones(5, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    mc, vc = torch.zeros(N, dtype=torch.int8, device=DEV), torch.zeros(N, dtype=torch.uint8, device=DEV)
    mq, vq = torch.zeros(N // 256, device=DEV), torch.zeros(N // 256, device=DEV)
    where = [0, (1 << 31) - 300, (1 << 32) - 300, n - 600]
    rng = np.random.default_rng(4)
    for a in where:
        g[a:a + 600] = torch.from_numpy(rng.standard_normal(600) * 1e-3).to(DEV).bfloat16()
    ctl = ob.control_create(DEV)
    ob.ob_grad_norm(lst, [small[0], g], ctl)
    hp = hparams(step=1)
    ob.ob_adamw8_step(lst, [small[0], g], [small[1], p], mc, mq, vc, vq, hp)
    torch.cuda.synchronize()
    s = float(g.float().square().sum(dtype=torch.float64)) + 5.0
    norm = float(ob.control_fields(ctl)["norm"])
    assert abs(norm - np.sqrt(s)) <= EPS32 * np.sqrt(s)   # the library's fp32 squares add 2^-24 at most
    for a in where:
        a0, a1 = a // 256 * 256, min(n, (a + 600 + 255) // 256 * 256)
        x = f64(g[a0:a1])
        m, v = ref.adamw8_moments(x, 0 * x, 0 * x, beta1=hp.beta1, beta2=hp.beta2)
        for y, second, c, q in ((m, False, mc, mq), (v, True, vc, vq)):
            wc, wq = ref.encode(y, second)
            assert np.array_equal(c[o + a0:o + a1].cpu().numpy(), wc), a
            assert np.array_equal(q[(o + a0) // 256:][: len(wq)].cpu().numpy(), wq), a
        u = (m / ref.bc(hp.beta1, 1)) / (np.sqrt(v / ref.bc(hp.beta2, 1)) + 1e-8)
        want = 0.5 - float(hp.lr) * (u + float(hp.weight_decay) * 0.5)
        close(f64(p[a0:a1]), want, 2.0 ** -8 * np.abs(want), a)


def test_huge_tensor_with_fp32_states():
    """Offsets past 2^31 elements: the places around it and the end."""
    n = (1 << 31) + 4099
    lst = ob.ob_tensors_create([5, n], torch.bfloat16, torch.float32)
    N, o = lst.state_elems, lst.state_offset(1)
    g = torch.full((n,), 1e-3, dtype=torch.bfloat16, device=DEV)
    p = torch.full((n,), 0.5, device=DEV)
    m, v = torch.zeros(N, device=DEV), torch.zeros(N, device=DEV)
    where = [0, (1 << 31) - 300, n - 600]
    rng = np.random.default_rng(4)
    for a in where:
        g[a:a + 600] = torch.from_numpy(rng.standard_normal(600) * 1e-3).to(DEV).bfloat16()
    hp = hparams(step=1)
    ob.ob_adamw_step(lst, [None, g], [None, p], m, v, hp)
    for a in where:
        x = f64(g[a:a + 600])
        wm, wv, wp, u = ref.adamw(x, 0 * x, 0 * x, 0 * x + 0.5, lr=float(hp.lr), beta1=hp.beta1, beta2=hp.beta2, eps=hp.eps,
                                  wd=float(hp.weight_decay), bc1=ref.bc(hp.beta1, 1), bc2=ref.bc(hp.beta2, 1))
        for got, want in ((m[o + a:o + a + 600], wm), (v[o + a:o + a + 600], wv), (p[a:a + 600], wp)):
            close(f64(got), want, EPS32 / 2 * np.abs(want) * (1 + 1e-6) + 2.0 ** -46 * np.abs(float(hp.lr) * u), a)
    assert not m[:o].any() and not v[:o].any()


def test_huge_conversion():
    n = (1 << 31) + 300
    x = torch.zeros(n, device=DEV)
    c, q = torch.zeros(n, dtype=torch.int8, device=DEV), torch.zeros(-(-n // 256), device=DEV)
    where = [0, (1 << 31) - 256, n // 256 * 256 - 256]
    rng = np.random.default_rng(6)
    tail = n - where[-1]
    parts = [rng.standard_normal(k).astype(np.float32) for k in (512, 256, tail)]
    for a, y in zip(where, parts):
        x[a:a + len(y)] = torch.from_numpy(y).to(DEV)
    ob.ob_state8_encode(x, None, c, q, None, None)
    x.zero_()
    ob.ob_state8_decode(c, q, None, None, x, None)
    for a, y in zip(where, parts):
        wc, wq = ref.encode(y, False)
        assert np.array_equal(c[a:a + len(y)].cpu().numpy(), wc) and np.array_equal(q[a // 256:][: len(wq)].cpu().numpy(), wq)
        assert np.array_equal(f64(x[a:a + len(y)]), ref.decode(wc, wq, False))


# ---- the norm and the control block ----

@pytest.mark.parametrize("g", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("sizes", [[1], [0, 3], SIZES, [70_001, 5, 2_000_003], [7] * 1500], ids=lambda s: f"{len(s)}tensors")
def test_norm(g, sizes):
    L = Lists(sizes, g, "f32", seed=12)
    ctl = ob.control_create(DEV)
    f = ob.control_fields(ctl)
    for g_mult, max_norm in ((1.0, 0.0), (1.0, 1e-3), (-0.25, 1e6), (1.0 / 1024, float("inf"))):
        ob.ob_grad_norm(L.list, L.grads, ctl, g_mult, max_norm)
        norm, factor = ref.grad_norm([f64(x) for x in L.grads], g_mult, max_norm)
        assert abs(float(f["norm"]) - norm) <= EPS32 / 2 * (1 + 1e-6) * norm
        assert abs(float(f["grad_scale"]) - factor) <= EPS32 / 2 * (1 + 1e-6) * abs(factor)
        assert int(f["skip"]) == 0 and int(f["step"]) == 0
    bits = ctl[:2].clone()
    for _ in range(5):
        ob.ob_grad_norm(L.list, L.grads, ctl, g_mult, max_norm)
        assert torch.equal(ctl[:2], bits)
    L.check_guards()


def test_norm_of_mixed_types_and_missing_gradients():
    rng = np.random.default_rng(1)
    T = 1000
    kinds = ["f32", "bf16", "f16"]
    L = Lists([int(x) for x in rng.integers(0, 3000, T)], [kinds[i] for i in rng.integers(0, 3, T)], "f32", seed=2)
    L.draw_grads(set(range(0, T, 3)))
    ctl = ob.control_create(DEV)
    ob.ob_grad_norm(L.list, L.grads, ctl)
    norm, _ = ref.grad_norm([None if x is None else f64(x) for x in L.grads], 1.0, 0.0)
    assert abs(float(ob.control_fields(ctl)["norm"]) - norm) <= EPS32 / 2 * (1 + 1e-6) * norm
    L.draw_grads(set(range(T)))   # nothing at all: norm 0, no factor below 1
    ob.ob_grad_norm(L.list, L.grads, ctl, 1.0, 1.0)
    f = ob.control_fields(ctl)
    assert float(f["norm"]) == 0.0 and float(f["grad_scale"]) == 1.0


def test_norm_of_large_values_does_not_overflow():
    L = Lists([1000], "f32", "f32", seed=2, shift=False)
    L.grads[0].fill_(1e30)
    ctl = ob.control_create(DEV)
    ob.ob_grad_norm(L.list, L.grads, ctl, 1.0, 1.0, hparams())
    f = ob.control_fields(ctl)
    want = np.sqrt(1000.0) * float(np.float32(1e30))
    assert abs(float(f["norm"]) - want) <= EPS32 / 2 * (1 + 1e-6) * want and int(f["skip"]) == 0


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_step_is_left_out_when_the_norm_is_not_finite(bits, bad):
    L = Lists([300, 5000], "bf16", "bf16", seed=4, bits=bits, master=True)
    ctl = ob.control_create(DEV)
    f = ob.control_fields(ctl)
    hp = hparams()
    L.grads[1][4999] = bad
    before = L.snapshot()
    ob.ob_grad_norm(L.list, L.grads, ctl, 1.0, 1.0, hp)
    L.step(hp, ctl)
    torch.cuda.synchronize()
    after = L.snapshot()
    assert int(f["skip"]) == 1 and int(f["skipped"]) == 1 and int(f["step"]) == 0
    for a, b in zip(before["p"] + [before["m"], before["v"], before["master"]], after["p"] + [after["m"], after["v"], after["master"]]):
        assert np.array_equal(a, b)
    L.draw_grads()
    ob.ob_grad_norm(L.list, L.grads, ctl, 1.0, 1.0, hp)
    L.step(hp, ctl)
    torch.cuda.synchronize()
    assert int(f["skip"]) == 0 and int(f["skipped"]) == 1 and int(f["step"]) == 1
    L.check(before, hp, t=1, scale=float(f["grad_scale"]))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("stochastic", [False, True])
def test_norm_step_and_moments_together(bits, stochastic):
    """A loop as a program runs it: loss-scaled fp16 gradients, clipping, a rate schedule, parameter groups; then the
    moments read back in fp32."""
    L = Lists([4096, 10, 777, 12_345], "f16", "bf16", seed=6, bits=bits, lr_mults=[1.0, 0.1, 1.0, 2.0],
              wd_mults=[1.0, 0.0, 1.0, 1.0], grad_sigma=0.5)
    ctl = ob.control_create(DEV)
    f = ob.control_fields(ctl)
    for t in range(1, 5):
        hp = hparams(rounding=int(stochastic), sr_seed=77)
        f["lr_scale"].fill_(0.25 * t)
        before = L.snapshot()
        ob.ob_grad_norm(L.list, L.grads, ctl, 1 / 512, 0.05, hp)
        L.step(hp, ctl)
        torch.cuda.synchronize()
        norm, factor = ref.grad_norm([f64(x) for x in L.grads], 1 / 512, 0.05)
        assert abs(float(f["norm"]) - norm) <= EPS32 / 2 * (1 + 1e-6) * norm and norm > 0.05
        assert int(f["step"]) == t
        assert abs(float(f["bc1"]) - ref.bc(0.9, t)) <= 1e-14 and abs(float(f["bc2"]) - ref.bc(0.98, t)) <= 1e-14
        after = L.check(before, hp, t=t, scale=float(f["grad_scale"]), lr_scale=0.25 * t)
        L.draw_grads()
    if bits == 8:
        m, v = torch.empty(L.N, device=DEV), torch.empty(L.N, device=DEV)
        ob.ob_state8_decode(L.mc, L.mq, L.vc, L.vq, m, v)
        assert np.array_equal(f64(m)[L.inside], after["m"][L.inside])
        assert np.array_equal(f64(v)[L.inside], after["v"][L.inside])


# ---- the 8-bit format ----

@pytest.mark.parametrize("n", [1, 3, 4, 255, 256, 257, 1000, 4096, 4097, 100_003])
def test_encode_and_decode(n):
    rng = np.random.default_rng(n)
    m = (rng.standard_normal(n) * 10.0 ** rng.uniform(-8, 0, n)).astype(np.float32)
    v = (rng.standard_normal(n) ** 2 * 10.0 ** rng.uniform(-16, 0, n)).astype(np.float32)
    if n > 4000:
        m[10], m[11], v[12], v[20] = 0, -0.0, 0, -0.0
        m[256:512] = 0
        m[512:768], v[512:768] = 1e-30, 1e-30        # below 2^-96: zeros
        m[800], v[801] = np.nan, np.inf
        m[1100], v[1100] = -np.inf, -1e-5            # a negative v reads as NaN
        v[1300:1400] = 1e-40
        v[1536:1792] = 2.0 ** -96
        m[1792:2048] = 3e38
        v[1792:2048] = 3e38
        k = np.arange(1, 128)                        # on and beside the borders of codes
        q = np.float32(3e-4)
        edge = ((k - 0.5) ** 2 * float(q)).astype(np.float32)
        m[2048:2048 + 127], m[2180:2180 + 120] = edge, np.nextafter(edge[:120], np.float32(0))
        m[2303] = 16129 * q
    G = 64
    buf = {k: torch.full((n + G,), 77, dtype=d, device=DEV) for k, d in (("mc", torch.int8), ("vc", torch.uint8))}
    mq, vq = torch.full((-(-n // 256) + 4,), 7.0, device=DEV), torch.full((-(-n // 256) + 4,), 7.0, device=DEV)
    nb = -(-n // 256)
    args = buf["mc"][:n], mq[:nb], buf["vc"][:n], vq[:nb]
    ob.ob_state8_encode(torch.from_numpy(m).to(DEV), torch.from_numpy(v).to(DEV), *args)
    torch.cuda.synchronize()
    for x, second, c, q in ((m, False, "mc", mq), (v, True, "vc", vq)):
        wc, wq = ref.encode(x, second)
        assert np.array_equal(q[:nb].cpu().numpy(), wq, equal_nan=True)
        assert np.array_equal(buf[c][:n].cpu().numpy(), wc)
        assert torch.all(buf[c][n:] == 77) and torch.all(q[nb:] == 7.0)
    out = [torch.full((n + G,), 7.0, device=DEV) for _ in range(2)]
    ob.ob_state8_decode(*args, out[0][:n], out[1][:n])
    for x, second, y in ((m, False, out[0]), (v, True, out[1])):
        want = ref.decode(*ref.encode(x, second), second)
        assert np.array_equal(f64(y)[:n], want, equal_nan=True)
        assert torch.all(y[n:] == 7.0)
    # one moment without the other
    c2, q2 = torch.empty(n, dtype=torch.int8, device=DEV), torch.empty(nb, device=DEV)
    ob.ob_state8_encode(torch.from_numpy(m).to(DEV), None, c2, q2, None, None)
    assert torch.equal(c2, args[0])
    c3, q3 = torch.empty(n, dtype=torch.uint8, device=DEV), torch.empty(nb, device=DEV)
    ob.ob_state8_encode(None, torch.from_numpy(v).to(DEV), None, None, c3, q3)
    assert torch.equal(c3, args[2])
    y = torch.empty(n, device=DEV)
    ob.ob_state8_decode(None, None, c3, q3, None, y)
    assert torch.equal(y.view(torch.int32), out[1][:n].view(torch.int32))


# ---- streams, graphs, overlapping calls ----

def _run_loop(L, ctl, hp, grads, step):
    out = []
    for gs in grads:
        for x, y in zip(L.grads, gs):
            x.copy_(y)
        step()
        torch.cuda.synchronize()
        out.append([x.clone() for x in L.params + [L.mc, L.mq, L.vc, L.vq, L.master, ctl[:12]]])
    return out


def test_graph_replays_are_eager_steps():
    """Norm and step captured once and replayed with new gradients and rates, with eager work between replays."""
    hp = hparams(rounding=1, sr_seed=5)
    runs = []
    for captured in (False, True):
        L = Lists([5000, 3, 70_000], "bf16", "bf16", seed=21, bits=8, master=True)
        ctl = ob.control_create(DEV)
        rng = np.random.default_rng(5)
        grads = [[torch.from_numpy(rng.standard_normal(n) * 1e-3).to(DEV).bfloat16() for n in L.sizes] for _ in range(4)]

        def call():
            ob.ob_grad_norm(L.list, L.grads, ctl, 1.0, 0.1, hp)
            L.step(hp, ctl)

        if captured:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                call()
            torch.cuda.synchronize()

        def step():
            ob.control_fields(ctl)["lr_scale"].mul_(0.9)
            torch.cuda.synchronize()
            graph.replay() if captured else call()

        runs.append(_run_loop(L, ctl, hp, grads, step))
    for a, b in zip(*runs):
        for x, y in zip(a, b):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_two_streams_share_a_list():
    """A list holds no workspace: two programs step their own buffers through one list at once, each with the results that it
    has alone."""
    hp = hparams()
    a, b = (Lists([200_000, 77, 1_000_003], "bf16", "f32", seed=s, bits=8) for s in (1, 2))
    alone = []
    for L in (a, b):
        keep = [x.clone() for x in L.params + [L.mc, L.mq, L.vc, L.vq]]
        ctl = ob.control_create(DEV)
        for _ in range(10):
            ob.ob_grad_norm(a.list, L.grads, ctl, 1.0, 0.1, hp)
            ob.ob_adamw8_step(a.list, L.grads, L.params, L.mc, L.mq, L.vc, L.vq, hp, None, ctl)
        torch.cuda.synchronize()
        alone.append([x.clone() for x in L.params + [L.mc, L.mq, L.vc, L.vq]])
        for x, y in zip(L.params + [L.mc, L.mq, L.vc, L.vq], keep):
            x.copy_(y)
    streams, ctls = [torch.cuda.Stream() for _ in range(2)], [ob.control_create(DEV) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for L, s, ctl in zip((a, b), streams, ctls):
            ob.ob_grad_norm(a.list, L.grads, ctl, 1.0, 0.1, hp, stream=s)
            ob.ob_adamw8_step(a.list, L.grads, L.params, L.mc, L.mq, L.vc, L.vq, hp, None, ctl, stream=s)
    torch.cuda.synchronize()
    for L, want in zip((a, b), alone):
        for x, y in zip(L.params + [L.mc, L.mq, L.vc, L.vq], want):
            assert torch.equal(x, y)


# ---- refusals ----

def test_refusals():
    L = Lists([300, 5], "bf16", "bf16", seed=1, bits=8)
    hp, ctl = hparams(), ob.control_create(DEV)
    call = lambda **kw: ob.ob_adamw8_step(**{**dict(tensors=L.list, grads=L.grads, params=L.params, m_codes=L.mc, m_scales=L.mq,  # noqa: E731
                                                    v_codes=L.vc, v_scales=L.vq, hp=hp), **kw})
    before = L.snapshot()
    with pytest.raises(ValueError, match="2 tensors"):
        call(grads=L.grads[:1])
    with pytest.raises(TypeError, match=r"grads\[1\]"):
        call(grads=[L.grads[0], L.grads[1].float()])
    with pytest.raises(ValueError, match=r"params\[0\]"):
        call(params=[L.params[0][:299], L.params[1]])
    with pytest.raises(ValueError, match="contiguous"):
        call(grads=[torch.zeros(600, dtype=torch.bfloat16, device=DEV)[::2], L.grads[1]])
    with pytest.raises(ValueError, match="GPU"):
        call(grads=[L.grads[0].cpu(), L.grads[1]])
    with pytest.raises(TypeError, match=r"params\[1\]"):
        call(params=[L.params[0], None])
    with pytest.raises(TypeError, match="m_codes"):
        call(m_codes=L.vc)
    with pytest.raises(ValueError, match="v_scales"):
        call(v_scales=L.vq[:1])
    with pytest.raises(ValueError, match="control"):
        call(control=ctl[:16])
    with pytest.raises(ValueError, match="control"):
        ob.ob_grad_norm(L.list, L.grads, ctl[:16])
    with pytest.raises(ValueError, match=r"m_codes must be on the GPU"):
        call(m_codes=L.mc.cpu())
    with pytest.raises(TypeError, match=r"grads\[0\]"):
        call(grads=[3, L.grads[1]])
    with pytest.raises(ValueError, match="dense"):
        call(grads=[torch.zeros(300, dtype=torch.bfloat16, device=DEV).to_sparse(), L.grads[1]])
    with pytest.raises(TypeError, match="adamw_hparams"):
        call(hp=ob.hparams())
    with pytest.raises(TypeError):
        ob.ob_grad_norm(L.list, L.grads, ctl, "1")
    with pytest.raises(TypeError):
        ob.ob_grad_norm(L.list, L.grads, ctl[:16], "1")
    with pytest.raises(ValueError, match="destroyed"):
        gone = ob.ob_tensors_create([300, 5], torch.bfloat16, torch.bfloat16)
        gone.destroy()
        call(tensors=gone)
    with pytest.raises(ob.ObError) as e:
        call(params=[L.params[0], L.params[0][10:15]])   # one parameter inside another
    assert e.value.status == 1
    for bad in (dict(beta1=1.0), dict(eps=0.0), dict(step=0), dict(rounding=5), dict(lr=float("nan"))):
        with pytest.raises(ob.ObError):
            call(hp=hparams(**bad))
    with pytest.raises(ob.ObError):
        ob.ob_grad_norm(L.list, L.grads, ctl, 0.0)
    with pytest.raises(ob.ObError) as e:
        ob.ob_state8_encode(torch.zeros(301, device=DEV)[1:], None, torch.zeros(300, dtype=torch.int8, device=DEV),
                            torch.zeros(2, device=DEV), None, None)
    assert e.value.status == 2
    # straight to the C ABI: missing states and addresses
    g, p = ((ctypes.c_void_p * 2)(*[t.data_ptr() for t in x]) for x in (L.grads, L.params))
    lib, P = ob.lib(), ctypes.c_void_p
    h = ctypes.byref(hp)
    assert lib.ob_adamw_step(L.list.handle, g, p, None, None, P(0x1000), h, None, None) == 1
    assert lib.ob_adamw_step(L.list.handle, g, p, None, P(0x1004), P(0x1000), h, None, None) == 2
    assert lib.ob_adamw8_step(L.list.handle, g, p, None, P(0x1000), None, P(0x1000), P(0x1000), h, None, None) == 1
    assert lib.ob_adamw8_step(L.list.handle, g, p, None, P(0x1002), P(0x1000), P(0x1000), P(0x1000), h, None, None) == 2
    assert lib.ob_grad_norm(L.list.handle, g, 1.0, 1.0, None, None, None) == 1
    torch.cuda.synchronize()
    after = L.snapshot()
    assert all(np.array_equal(x, y) for x, y in zip(before["p"], after["p"])) and np.array_equal(before["mc"], after["mc"])


def test_tensors_without_their_memory_are_refused():
    """A released storage has no address, which would read as an argument left out; a shrunk one ends too early.  All
    are refused on the host, before a launch."""
    def gone(like, nbytes=0):
        t = like.clone()
        t.untyped_storage().resize_(nbytes)
        return t

    for bits in (32, 8):
        L = Lists([300, 5], "bf16", "bf16", seed=1, bits=bits, master=True)
        hp, ctl = hparams(), ob.control_create(DEV)
        states = dict(m=L.m, v=L.v) if bits == 32 else dict(m_codes=L.mc, m_scales=L.mq, v_codes=L.vc, v_scales=L.vq)
        good = dict(tensors=L.list, grads=L.grads, params=L.params, hp=hp, master=L.master, control=ctl, **states)
        step = ob.ob_adamw_step if bits == 32 else ob.ob_adamw8_step
        tensors = [*L.params, L.master, *states.values()]
        before = [t.clone() for t in tensors]
        for nbytes in (0, 4):
            for k in ("master", "control", *states):
                with pytest.raises(ValueError, match=f"{k} must have its memory"):
                    step(**{**good, k: gone(good[k], nbytes)})
            for k in ("grads", "params"):
                with pytest.raises(ValueError, match=rf"{k}\[0\] must have its memory"):
                    step(**{**good, k: [gone(good[k][0], nbytes), good[k][1]]})
            with pytest.raises(ValueError, match=r"grads\[1\] must have its memory"):
                ob.ob_grad_norm(L.list, [L.grads[0], gone(L.grads[1], nbytes)], ctl)
            with pytest.raises(ValueError, match="control must have its memory"):
                ob.ob_grad_norm(L.list, L.grads, gone(ctl, nbytes))
        for t, b in zip(tensors, before):
            assert torch.equal(t, b)
    x = torch.zeros(300, device=DEV)
    codes, scales = torch.zeros(300, dtype=torch.int8, device=DEV), torch.zeros(2, device=DEV)
    for call in (lambda: ob.ob_state8_encode(gone(x), None, codes, scales, None, None),
                 lambda: ob.ob_state8_decode(codes, gone(scales), None, None, x, None)):
        with pytest.raises(ValueError, match="must have its memory"):
            call()


def test_empty_lists():
    hp, ctl = hparams(), ob.control_create(DEV)
    for sizes in ([], [0, 0]):
        lst = ob.ob_tensors_create(sizes, torch.float32, torch.float32)
        e = torch.zeros(0, device=DEV)
        ob.ob_grad_norm(lst, [e] * len(sizes), ctl, 1.0, 1.0, hp)
        ob.ob_adamw_step(lst, [e] * len(sizes), [e] * len(sizes), e, e, hp, None, ctl)
        assert float(ob.control_fields(ctl)["norm"]) == 0.0 and len(lst) == len(sizes) and lst.state_elems == 0
    assert int(ob.control_fields(ctl)["step"]) == 2
    lst.destroy()
    lst.destroy()


# ---- the driver ----

def _model(dtype, seed=0):
    torch.manual_seed(seed)
    net = torch.nn.Sequential(torch.nn.Linear(33, 65), torch.nn.LayerNorm(65), torch.nn.GELU(), torch.nn.Linear(65, 7))
    return net.to(DEV).to(dtype)


def _train(net, opt, steps, seed=0, scale=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    for _ in range(steps):
        x = torch.randn(16, 33, generator=gen, device=DEV).to(next(net.parameters()).dtype)
        for p in net.parameters():
            p.grad = None
        (net(x).float().square().mean() * scale).backward()
        opt.step(loss_scale=scale) if scale != 1.0 else opt.step()


def test_driver_against_torch():
    """Two parameter groups, clipping, 5 steps against torch's AdamW on the same gradients.  Both are off by some 2^-24 of
    p and 2^-21 of an update of at most 2 lr a step."""
    a, b = _model(torch.float32), _model(torch.float32)
    decay = lambda net: [p for p in net.parameters() if p.dim() > 1]  # noqa: E731
    plain = lambda net: [p for p in net.parameters() if p.dim() < 2]  # noqa: E731
    opt = ob.AdamW([{"params": decay(a)}, {"params": plain(a), "weight_decay": 0.0, "lr": 2e-3}], lr=1e-3, weight_decay=0.1,
                   max_norm=0.5)
    want = torch.optim.AdamW([{"params": decay(b)}, {"params": plain(b), "weight_decay": 0.0, "lr": 2e-3}], lr=1e-3,
                             weight_decay=0.1, foreach=False)
    gen = torch.Generator(device=DEV).manual_seed(3)
    for _ in range(5):
        for p, q in zip(a.parameters(), b.parameters()):
            q.grad = torch.randn(p.shape, generator=gen, device=DEV)
            p.grad = q.grad.clone()
        norm = torch.nn.utils.clip_grad_norm_(list(b.parameters()), 0.5)
        opt.step()
        want.step()
        assert abs(float(opt.norm) - float(norm)) <= 1e-6 * float(norm)
    assert opt.steps() == 5
    for p, q in zip(a.parameters(), b.parameters()):
        tol = 5 * (2.0 ** -23 * q.abs() + 2 * 2e-3 * 2.0 ** -20)
        assert torch.all((p - q).abs() <= tol)


@pytest.mark.parametrize("bits,dtype,master,rounding", [(32, "f32", False, "nearest"), (8, "f32", False, "nearest"),
                                                        (8, "bf16", True, "stochastic"), (32, "bf16", False, "stochastic"),
                                                        (8, "bf16", False, "stochastic")])
@pytest.mark.parametrize("max_norm", [None, 1.0])
def test_driver_resumes_bit_for_bit(bits, dtype, master, rounding, max_norm):
    kw = dict(lr=1e-2, state_bits=bits, master=master, rounding=rounding, max_norm=max_norm, sr_seed=9)
    a = _model(DT[dtype])
    opt = ob.AdamW(a.parameters(), **kw)
    _train(a, opt, 3)
    saved = {k: x.cpu() if isinstance(x, torch.Tensor) else x for k, x in opt.state_dict().items()}
    b = _model(DT[dtype], seed=1)
    b.load_state_dict(a.state_dict())
    again = ob.AdamW(b.parameters(), **kw)
    again.load_state_dict(saved)
    assert again.steps() == 3
    _train(a, opt, 3, seed=8)
    _train(b, again, 3, seed=8)
    for p, q in zip(a.parameters(), b.parameters()):
        assert torch.equal(p, q)
    for k, x in opt.state_dict().items():
        assert x == again.state_dict()[k] if not isinstance(x, torch.Tensor) else torch.equal(x, again.state_dict()[k]), k


def test_driver_changes_width():
    a = _model(torch.float32)
    wide = ob.AdamW(a.parameters(), lr=1e-3)
    _train(a, wide, 4)
    narrow = ob.AdamW(a.parameters(), lr=1e-3, state_bits=8)
    narrow.load_state_dict(wide.state_dict())
    m, v = narrow.moments()
    for x, y, second in ((wide.m, m, False), (wide.v, v, True)):
        want = ref.decode(*ref.encode(x.cpu().numpy(), second), second)
        assert np.array_equal(f64(y), want)
    back = ob.AdamW(a.parameters(), lr=1e-3)
    back.load_state_dict(narrow.state_dict())
    assert torch.equal(back.m, m) and torch.equal(back.v, v) and back.steps() == 4


def test_driver_in_a_captured_step(monkeypatch):
    """The driver's step captured and replayed with new gradients and rates, against the same steps run eagerly."""
    nets = []
    for captured in (False, True):
        net = _model(torch.float32)
        opt = ob.AdamW(net.parameters(), lr=1e-3, state_bits=8, max_norm=float("inf"))
        for p in net.parameters():
            p.grad = torch.zeros_like(p)
        if captured:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                opt.step()
            torch.cuda.synchronize()
        gen = torch.Generator(device=DEV).manual_seed(4)
        for k in range(4):
            for p in net.parameters():
                p.grad.copy_(torch.randn(p.shape, generator=gen, device=DEV))
            opt.set_lr_scale(1.0 / (k + 1))
            torch.cuda.synchronize()
            graph.replay() if captured else opt.step()
            torch.cuda.synchronize()
        assert opt.steps() == 4
        nets.append([p.detach().clone() for p in net.parameters()])
    for p, q in zip(*nets):
        assert torch.equal(p, q)
    counted = ob.AdamW(net.parameters())   # a step count on the host cannot be replayed
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(RuntimeError, match="captured"):
        counted.step()


def test_driver_refusals():
    net = _model(torch.float32)
    opt = ob.AdamW(net.parameters())
    with pytest.raises(ValueError, match="loss scale"):
        opt.step([torch.zeros_like(p) for p in net.parameters()], loss_scale=2.0)
    with pytest.raises(ValueError, match="tensors"):
        opt.step([])
    with pytest.raises(ValueError, match="contiguous"):
        ob.AdamW([torch.zeros(8, 8, device=DEV).t()[:4]])
    with pytest.raises(ValueError, match="weight_decay"):
        ob.AdamW([{"params": list(net.parameters()), "weight_decay": 0.1}], weight_decay=0.0)
    with pytest.raises(ValueError, match="elements"):
        opt.load_state_dict({**opt.state_dict(), "m": opt.m[:256]})
    with pytest.raises(ValueError, match="master"):
        opt.load_state_dict({**opt.state_dict(), "master": opt.m})
    # a forward before the step keeps what its backward needs: a step in between is noticed
    x = torch.randn(4, 33, device=DEV)
    y = net(x).sum()
    opt.step([torch.zeros_like(p) for p in net.parameters()])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


@pytest.mark.parametrize("max_norm", [None, 1.0])
@pytest.mark.parametrize("bits", [32, 8])
def test_driver_does_not_count_a_refused_step(bits, max_norm):
    a, b = _model(torch.float32), _model(torch.float32)
    first, second = (ob.AdamW(net.parameters(), lr=1e-2, state_bits=bits, max_norm=max_norm) for net in (a, b))
    for bad in ([p.half() for p in a.parameters()], [p.detach().cpu() for p in a.parameters()], []):
        with pytest.raises((TypeError, ValueError)):
            first.step(bad)
        assert first.steps() == 0
    _train(a, first, 2)
    _train(b, second, 2)
    assert first.steps() == second.steps() == 2
    for p, q in zip(a.parameters(), b.parameters()):
        assert torch.equal(p, q)


def _check_codes(L, g, hp, t, blocks):
    """The given state blocks of a list of one fp32 tensor after its first step, against the rule."""
    words = ref.philox_words(hp.sr_seed, t, L.N).reshape(-1, 256)[blocks]
    m, v = ref.adamw8_moments(g.reshape(-1, 256)[blocks].reshape(-1).astype(np.float64), 0.0, 0.0, beta1=hp.beta1, beta2=hp.beta2)
    where = torch.from_numpy(blocks).to(DEV)
    for x, second, c, q in ((m, False, L.mc, L.mq), (v, True, L.vc, L.vq)):
        codes, scales = ref.encode(x, second, words.reshape(-1))
        got = c.view(-1, 256)[where].cpu().numpy().reshape(-1)
        bad = np.nonzero(got != codes)[0]
        assert np.array_equal(q[where].cpu().numpy(), scales), (second, t)
        assert len(bad) == 0, (second, t, len(bad), x[bad][:4], scales[bad // 256][:4], words.reshape(-1)[bad][:4], got[bad][:4], codes[bad][:4])


def _first_step_by_chance(L, g, t, seed):
    """One step from zero moments in which they become g and fl(g^2)."""
    L.mc.zero_(), L.mq.zero_(), L.vc.zero_(), L.vq.zero_()
    L.grads = [torch.from_numpy(g).to(DEV)]
    hp = hparams(beta1=0.0, beta2=0.0, step=t, rounding=1, sr_seed=seed)
    L.step(hp)
    torch.cuda.synchronize()
    return hp


@pytest.mark.parametrize("second", [False, True])
@pytest.mark.parametrize("blocks,steps", [(4000, 12), (36_000, 4)])   # one and four state blocks per wave
def test_codes_by_chance_beside_whole_codes(blocks, steps, second):
    """Moments within 3 fp32 steps of a code's value, where the random bits are the 4 smallest or largest ones: the rule's
    code there depends on which side of the value a moment lies."""
    n = blocks * 256
    L = Lists([n], "f32", "f32", seed=31, bits=8, shift=False)
    rng = np.random.default_rng(31)
    top = rng.uniform(0.5, 2.0, blocks).astype(np.float32)
    if second:
        q = ref.r32(ref.r32(np.sqrt(ref.r32(top.astype(np.float64) ** 2))) * ref.r32(1 / 255 ** 2))
    else:
        q = ref.r32(top.astype(np.float64) * ref.r32(1 / 127 ** 2))
    for t in range(1, steps + 1):
        words = ref.philox_words(5, t, n)
        bits = words >> 16 if second else words & 0xFFFF
        at = np.nonzero(((bits < 4) | (bits > 65531)) & (np.arange(n) % 256 != 0))[0]
        k = rng.integers(1, 255 if second else 127, len(at))
        x = ref.code_value(k, q[at // 256], second).astype(np.float32)
        x = (x.view(np.int32) + rng.integers(-3, 4, len(at), dtype=np.int32)).view(np.float32)
        g = (rng.standard_normal(n) * 1e-3).astype(np.float32)
        g[::256] = top
        g[at] = np.sqrt(x.astype(np.float64)) if second else x * rng.choice(np.float32([-1, 1]), len(at))
        hp = _first_step_by_chance(L, g, t, 5)
        _check_codes(L, g, hp, t, np.unique(at // 256))


@pytest.mark.parametrize("blocks", [64, 40_000])   # one and four state blocks per wave
def test_codes_by_chance_of_subnormal_second_moments(blocks):
    """The smallest blocks that have a scale: largest v in [2^-96, 2^-92), the others subnormal, where some get code 2."""
    n = blocks * 256
    L = Lists([n], "f32", "f32", seed=32, bits=8, shift=False)
    rng = np.random.default_rng(32)
    v = 2.0 ** rng.uniform(-129, -125, n)
    v[::256] = 2.0 ** rng.uniform(-96, -92, blocks)
    g = np.sqrt(v).astype(np.float32)
    hp = _first_step_by_chance(L, g, 1, 6)
    assert int((L.vc == 2).sum()) > n // 64
    _check_codes(L, g, hp, 1, np.arange(64))


def test_words_by_chance_past_a_counter_of_32_bits():
    """fp32 states around state index 2^34, where the generator's counter passes 32 bits, in a work group that starts
    256 and 768 elements before: the words of the rule.  The tensors before have no gradient."""
    where = (1 << 34) - 256
    for first in (0, 512):
        lst = ob.ob_tensors_create([where - first, 4099 + first], torch.bfloat16, torch.bfloat16)
        o, n = lst.state_offset(1), 4099 + first
        assert o == where - first
        m, v = (torch.empty(lst.state_elems, device=DEV) for _ in range(2))   # 64 GiB each, written in the second tensor only
        m[o:], v[o:] = 0, 0
        rng = np.random.default_rng(3)
        x = torch.from_numpy(rng.standard_normal(n) * 0.05).to(DEV).bfloat16()
        g = torch.from_numpy(rng.standard_normal(n) * 1e-3).to(DEV).bfloat16()
        p = x.clone()
        hp = hparams(step=1, rounding=1, sr_seed=0xABCDEF0123456789)
        ob.ob_adamw_step(lst, [None, g], [None, p], m, v, hp)
        _, _, want, u = ref.adamw(f64(g), 0.0, 0.0, f64(x), lr=float(hp.lr), beta1=hp.beta1, beta2=hp.beta2, eps=hp.eps,
                                  wd=float(hp.weight_decay), bc1=ref.bc(hp.beta1, 1), bc2=ref.bc(hp.beta2, 1))
        tol = EPS32 / 2 * np.abs(want) * (1 + 1e-6) + 2.0 ** -46 * (np.abs(f64(x)) + np.abs(float(hp.lr) * u))
        lo, hi = (from16(oracle.to_format_sr(y.astype(np.float32), "bf16", hp.sr_seed, 1 | ref.PAR_STREAM, o), "bf16")
                  for y in (want - tol, want + tol))
        got = f64(p)
        bad = np.nonzero(~((got >= np.minimum(lo, hi)) & (got <= np.maximum(lo, hi))))[0]
        assert len(bad) == 0, (first, len(bad), bad[:5])
        del m, v
        torch.cuda.empty_cache()


def _refused_by_the_step_alone(net, opt):
    """Calls that a norm would take and the step refuses, each mended after it."""
    first = next(net.parameters())
    grads = [torch.ones_like(p) for p in net.parameters()]
    keep = first.data
    first.data = keep.half()                      # another type
    yield grads, (TypeError,)
    first.data = keep.clone()
    first.data.untyped_storage().resize_(0)       # released
    yield grads, (ValueError,)
    first.data = keep[:0]                         # another size
    yield grads, (ValueError,)
    first.data = keep
    if opt.state_bits == 8:
        state, opt.m_scales = opt.m_scales, opt.m_scales[:1]
        yield grads, (ValueError,)
        opt.m_scales = state
        opt.hp.eps = 0.0
        yield grads, (ob.ObError,)
        opt.hp.eps = 1e-8
    opt.hp.beta2 = 1.0
    yield grads, (ob.ObError,)
    opt.hp.beta2 = 0.999


@pytest.mark.parametrize("max_norm", [None, 1.0])
@pytest.mark.parametrize("bits", [32, 8])
def test_driver_does_not_count_a_step_that_only_the_step_refuses(bits, max_norm):
    a, b = _model(torch.float32), _model(torch.float32)
    first, second = (ob.AdamW(net.parameters(), lr=1e-2, state_bits=bits, max_norm=max_norm) for net in (a, b))
    for grads, errors in _refused_by_the_step_alone(a, first):
        before = None if max_norm is None else first.control.clone()
        with pytest.raises(errors):
            first.step(grads)
        assert first.steps() == 0 and (before is None or torch.equal(first.control, before))
    _train(a, first, 2)
    _train(b, second, 2)
    assert first.steps() == second.steps() == 2
    for p, q in zip(a.parameters(), b.parameters()):
        assert torch.equal(p, q)


def test_driver_does_not_count_a_step_of_parameters_in_each_other():
    flat = torch.zeros(1000, device=DEV)
    opt = ob.AdamW([flat[:600], flat[500:]], max_norm=1.0)
    with pytest.raises(ob.ObError):
        opt.step([torch.ones(600, device=DEV), torch.ones(500, device=DEV)])
    assert opt.steps() == 0 and not flat.any()


@pytest.mark.parametrize("bits", [32, 8])
def test_norm_and_step_in_one_call(bits):
    """norm=(g_mult, max_norm): the results of the two calls; refused as a whole."""
    hp = hparams(rounding=1, sr_seed=3)
    out = []
    for together in (False, True):
        L = Lists(SIZES, "bf16", "bf16", seed=9, bits=bits, grad_sigma=0.5)
        ctl = ob.control_create(DEV)
        states = dict(m=L.m, v=L.v) if bits == 32 else dict(m_codes=L.mc, m_scales=L.mq, v_codes=L.vc, v_scales=L.vq)
        call = dict(tensors=L.list, grads=L.grads, params=L.params, hp=hp, control=ctl, **states)
        step = ob.ob_adamw_step if bits == 32 else ob.ob_adamw8_step
        for _ in range(3):
            if together:
                step(**call, norm=(0.5, 0.1))
            else:
                ob.ob_grad_norm(L.list, L.grads, ctl, 0.5, 0.1, hp)
                step(**call)
        out.append([x.clone() for x in [*L.params, *states.values(), ctl[:16]]])
        if together:
            for bad in (dict(norm=(0.0, 1.0)), dict(norm=(1.0, float("nan"))), dict(params=[L.params[0]] * len(SIZES)),
                        dict(control=None)):
                with pytest.raises((ob.ObError, TypeError, ValueError)):
                    step(**{**call, "norm": (1.0, 1.0), **bad})
            assert torch.equal(ctl[:16], out[-1][-1])
    for x, y in zip(*out):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("bits", [32, 8])
def test_driver_resumes_its_schedule(bits):
    """The factor of the rate and the count of left-out steps are part of the state."""
    kw = dict(lr=1e-2, state_bits=bits, max_norm=1.0)
    a = _model(torch.float32)
    opt = ob.AdamW(a.parameters(), **kw)
    opt.step([torch.full_like(p, float("nan")) for p in a.parameters()])
    opt.set_lr_scale(0.3)
    _train(a, opt, 2)
    b = _model(torch.float32, seed=1)
    b.load_state_dict(a.state_dict())
    again = ob.AdamW(b.parameters(), **kw)
    again.load_state_dict(opt.state_dict())
    f = ob.control_fields(again.control)
    assert float(f["lr_scale"]) == np.float32(0.3) and int(f["skipped"]) == 1 and again.steps() == 2
    _train(a, opt, 2, seed=8)
    _train(b, again, 2, seed=8)
    for p, q in zip(a.parameters(), b.parameters()):
        assert torch.equal(p, q)
    # a state without them leaves both; one with a factor needs a control block to hold it
    older = {k: x for k, x in opt.state_dict().items() if k not in ("lr_scale", "skipped")}
    again.load_state_dict(older)
    assert float(f["lr_scale"]) == np.float32(0.3) and int(f["skipped"]) == 1
    host = ob.AdamW(b.parameters(), lr=1e-2, state_bits=bits)
    host.load_state_dict(older)
    with pytest.raises(ValueError, match="max_norm"):
        host.load_state_dict(opt.state_dict())
    opt.set_lr_scale(1.0)
    host.load_state_dict(opt.state_dict())
    assert host.steps() == 4


def test_driver_takes_a_group_of_one_tensor():
    """A group's "params" may be a tensor; it is one parameter, not its rows."""
    a, b = (torch.nn.Parameter(torch.ones(7, 300, device=DEV)) for _ in range(2))
    for p, params in ((a, [{"params": a}]), (b, [{"params": [b]}])):
        opt = ob.AdamW(params)
        assert len(opt.params) == 1 and opt.params[0] is p
        p.grad = torch.full_like(p, 0.5)
        opt.step()
    assert torch.equal(a, b) and not torch.any(a == 1)


def test_driver_refuses_to_leave_out_what_is_no_leaf():
    """Rows of a parameter get no .grad of their own; with gradients given to the step they are stepped."""
    w = torch.nn.Parameter(torch.ones(2, 300, device=DEV))
    rows = list(w)
    opt = ob.AdamW(rows)
    w.grad = torch.ones_like(w)
    with pytest.raises(ValueError, match="leaf"):
        opt.step()
    assert opt.steps() == 0 and torch.all(w == 1)
    opt.step([torch.ones(300, device=DEV) for _ in rows])
    assert opt.steps() == 1 and not torch.any(w == 1)
    for x in rows:   # set by hand
        x.grad = torch.ones(300, device=DEV)
    opt.step()
    assert opt.steps() == 2
    kept = (torch.nn.Parameter(torch.ones(300, device=DEV)) * 1)
    kept.retain_grad()
    opt = ob.AdamW([kept])
    kept.sum().backward()
    opt.step()
    assert not torch.any(kept == 1)


def test_driver_looks_at_its_own_stream_for_a_capture(monkeypatch):
    """A step counted on the host is refused where the stream that it is given is being captured."""
    net = _model(torch.float32)
    opt = ob.AdamW(net.parameters())
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: torch.cuda.current_stream().cuda_stream == s.cuda_stream)
    grads = [torch.ones_like(p) for p in net.parameters()]
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        with pytest.raises(RuntimeError, match="captured"):
            opt.step(grads, stream=stream)
    assert opt.steps() == 0
    for stream in (other, other.cuda_stream, 0):
        opt.step(grads, stream=stream)
    with torch.cuda.stream(s):
        opt.step(grads, stream=other)
        with pytest.raises(RuntimeError, match="captured"):
            opt.step(grads)
    assert opt.steps() == 4
    torch.cuda.synchronize()


def test_driver_loads_a_whole_state_or_nothing():
    net = _model(torch.float32)
    narrow, wide = (ob.AdamW(net.parameters(), state_bits=bits, max_norm=1.0) for bits in (8, 32))
    for opt in (narrow, wide):
        _train(net, opt, 2)
    for opt, other in ((narrow, wide), (wide, narrow)):
        for d in (opt.state_dict(), other.state_dict()):
            d = {k: x.clone() + 1 if isinstance(x, torch.Tensor) else x for k, x in d.items()}
            d["step"] = 7
            before = {k: x.clone() if isinstance(x, torch.Tensor) else x for k, x in opt.state_dict().items()}
            for k in d:
                if k in ("lr_scale", "skipped"):
                    continue
                cut = {j: x for j, x in d.items() if j != k}
                bad = {**d, k: d[k].double().cpu() if isinstance(d[k], torch.Tensor) else "x"}
                bad = [cut] if isinstance(d[k], torch.Tensor) and d["state_bits"] == opt.state_bits else [cut, bad]
                for b in bad:
                    with pytest.raises((ValueError, TypeError), match=k):
                        opt.load_state_dict(b)
                    for j, x in opt.state_dict().items():
                        assert torch.equal(x, before[j]) if isinstance(x, torch.Tensor) else x == before[j], (k, j)


def test_driver_has_a_rate_factor_with_max_norm_only():
    opt = ob.AdamW(_model(torch.float32).parameters())
    with pytest.raises(ValueError, match="max_norm"):
        opt.set_lr_scale(0.5)
