"""CPU checks of the steps over lists of tensors: the host side (layout, work blocks, launches, refusals), the
binding's refusals, and the references that the GPU tests compare with."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import _adamw_ref as ref
import adam_ob_compress_amd as ob
import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_host_side_of_lists(tmp_path):
    exe = str(tmp_path / "list_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-D__HIP_PLATFORM_AMD__", "-I",
                    os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "adam_ob_compress_amd", "csrc"), "-I",
                    "/opt/rocm/include", os.path.join(ROOT, "tests", "list_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok 140"), r.stdout


def test_layouts_match_the_header():
    # five floats and an int32, an 8-byte aligned int64, two int32, uint64
    assert ctypes.sizeof(ob.ob_adamw_hparams) == 48
    assert ob.ob_adamw_hparams.step.offset == 24 and ob.ob_adamw_hparams.sr_seed.offset == 40
    c = torch.zeros(ob.OB_CONTROL_BYTES // 4, dtype=torch.int32)
    f = ob.control_fields(c)
    for name, at in (("norm", 0), ("grad_scale", 4), ("step", 8), ("skipped", 16), ("bc1", 24), ("bc2", 32),
                     ("lr_scale", 40), ("skip", 44)):
        assert f[name].data_ptr() - c.data_ptr() == at, name


def test_null_handles_are_refused():
    lib = ob.lib()
    hp = ob.adamw_hparams()
    P = ctypes.c_void_p
    assert lib.ob_tensors_create(1, None, None, None, None, None, None) == ob._native.OB_ERR_ARG
    h = P(1)
    sizes = (ctypes.c_int64 * 1)(-5)
    types = (ctypes.c_int32 * 1)(0)
    assert lib.ob_tensors_create(1, sizes, types, types, None, None, ctypes.byref(h)) == 1 and h.value is None
    types[0] = 7
    assert lib.ob_tensors_create(1, sizes, types, types, None, None, ctypes.byref(h)) == 3
    assert lib.ob_tensors_destroy(None) == 1
    for f in (lib.ob_tensors_count, lib.ob_tensors_num_elements, lib.ob_tensors_state_elems):
        assert f(None) == -1
    assert lib.ob_tensors_state_offset(None, 0) == -1
    assert lib.ob_grad_norm(None, None, 1.0, 1.0, None, P(0x1000), None) == 1
    assert lib.ob_adamw_step(None, None, None, None, None, None, ctypes.byref(hp), None, None) == 1
    assert lib.ob_adamw8_step(None, None, None, None, None, None, None, None, ctypes.byref(hp), None, None) == 1
    assert lib.ob_state8_encode(-1, None, None, None, None, None, None, None) == 1
    assert lib.ob_state8_decode(8, P(0x1000), None, None, None, P(0x2000), None, None) == 1
    assert lib.ob_state8_encode(0, None, None, None, None, None, None, None) == 0


def test_a_list_that_does_not_fit_the_host_is_a_status():
    """2^40 elements (2^28 work blocks, 4 GB of table) under a 4 GiB limit: OB_ERR_OOM, not an abort."""
    import sys
    code = f"""
import ctypes, resource
resource.setrlimit(resource.RLIMIT_AS, (4 << 30, 4 << 30))
L = ctypes.CDLL({ob.LIB_PATH!r})
h = ctypes.c_void_p(1)
n, d = (ctypes.c_int64 * 1)(1 << 40), (ctypes.c_int32 * 1)(0)
print(L.ob_tensors_create(ctypes.c_int64(1), n, d, d, None, None, ctypes.byref(h)), h.value)
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split() == [str(ob.OB_ERR_OOM), "None"]


def test_binding_refuses_host_tensors():
    x = torch.zeros(300)
    with pytest.raises(ValueError, match="GPU"):
        ob.ob_tensors_create([4], torch.float32, torch.float32, device="cpu")
    with pytest.raises(TypeError, match="g_dtype"):
        ob.ob_tensors_create([4], torch.float64, torch.float32)
    with pytest.raises(ValueError, match="entries"):
        ob.ob_tensors_create([4, 5], [torch.float32], torch.float32)
    c, q = torch.zeros(300, dtype=torch.int8), torch.zeros(2)
    with pytest.raises(ValueError, match="GPU"):
        ob.ob_state8_encode(x, None, c, q, None, None)
    with pytest.raises(ValueError, match="come together"):
        ob.ob_state8_encode(x, None, c, None, None, None)
    with pytest.raises(ValueError, match="elements"):
        ob.ob_state8_decode(c, q[:1], None, None, x, None)
    with pytest.raises(ValueError):
        ob.AdamW([])
    with pytest.raises(ValueError):
        ob.AdamW([x], state_bits=4)
    with pytest.raises(ValueError, match="twice"):
        ob.AdamW([x, x])
    with pytest.raises(ValueError, match="GPU"):
        ob.AdamW([x])


# ---- the references ----

def test_reference_random_words_are_the_oracles():
    seed, t = 0x123456789ABCDEF, 0x8000000000000123
    w = ref.philox_words(seed, t, 1001)
    for i in (0, 1, 2, 3, 4, 517, 1000):
        want = oracle.philox4x32([i >> 2, 0, t & 0xFFFFFFFF, t >> 32], [seed & 0xFFFFFFFF, seed >> 32])
        assert w[i] == want[i & 3]


@pytest.mark.parametrize("second", [False, True])
def test_reference_format(second):
    """Every code of a block comes back as itself, values are in order, the nearest code is within half a step
    in the companded scale, and the rules' special blocks hold."""
    most = 255 if second else 127
    k = np.arange(most + 1)
    x = ref.code_value(k, float(ref.r32(3e-4 / most ** 2)), second).astype(np.float32)
    assert np.all(np.diff(x) > 0)
    codes, scales = ref.encode(x, second)
    assert np.array_equal(codes, k)
    rng = np.random.default_rng(3)
    x = (rng.standard_normal(5000) * 10.0 ** rng.uniform(-9, 0, 5000)).astype(np.float32)
    x = x * x if second else x
    codes, scales = ref.encode(x, second)
    q = np.repeat(scales.astype(np.float64), 256)[: len(x)]
    root = np.sqrt(np.sqrt(np.abs(x.astype(np.float64)))) if second else np.sqrt(np.abs(x.astype(np.float64)))
    y = root / np.sqrt(q)
    off = np.abs(np.abs(codes.astype(np.float64)) - y)
    # half a step, and where a positive v is lifted to code 1 up to a whole one; 1e-4: the borders' fp32 rounding
    assert np.all(off <= np.where((codes == 1) & second, 1.0, 0.5) + 1e-4)
    assert np.array_equal(ref.decode(codes, scales, second)[x == 0], np.zeros(np.sum(x == 0)))
    x = np.zeros(1100, np.float32)
    x[300], x[600], x[1030] = 1e-30, np.inf, 2.0 ** -96
    codes, scales = ref.encode(x, second)
    assert scales[0] == 0 and scales[1] == 0 and np.isnan(scales[2]) and scales[3] == 0 and scales[4] > 0
    assert codes[1030] == most and not codes[:1030].any()
    if second:
        x = np.array([1.0, 1e-20, 0.0, -0.0], np.float32)
        assert ref.encode(x, True)[0].tolist() == [255, 1, 0, 0]
        assert np.isnan(ref.encode(np.array([1.0, -1e-3], np.float32), True)[1][0])


@pytest.mark.parametrize("second", [False, True])
def test_reference_chance_is_unbiased(second):
    """Mean over 4000 draws of one value between two codes: within 5 standard errors of it."""
    x = np.full(4096, 0.3, np.float32)
    x[::256] = 1.0
    codes, scales = ref.encode(x, second, ref.philox_words(99, 5, 4096))
    v = ref.decode(codes, scales, second)[x < 1]
    gap = v.max() - v.min()
    assert len(np.unique(v)) == 2 and v.min() < 0.3 < v.max()
    assert abs(v.mean() - np.float32(0.3)) < 5 * 0.5 * gap / np.sqrt(len(v)) + gap / 65536


def test_reference_step_is_torchs():
    """The fp64 lines against torch.optim.AdamW in fp64 over 5 steps (the reference rounds its moments to fp32 once a
    step: 2^-24 relative, which the update's line passes on one for one)."""
    rng = np.random.default_rng(1)
    p0 = rng.standard_normal(64)
    p = torch.nn.Parameter(torch.tensor(p0))
    f = lambda x: float(np.float32(x))  # noqa: E731
    opt = torch.optim.AdamW([p], lr=f(1e-2), betas=(f(0.9), f(0.99)), eps=f(1e-8), weight_decay=f(0.1))
    m = v = np.zeros(64)
    x = p0
    for t in range(1, 6):
        g = rng.standard_normal(64).astype(np.float32).astype(np.float64)
        p.grad = torch.tensor(g)
        opt.step()
        m, v, x, _ = ref.adamw(g, m, v, x, lr=f(1e-2), beta1=0.9, beta2=0.99, eps=1e-8, wd=f(0.1), bc1=ref.bc(0.9, t),
                               bc2=ref.bc(0.99, t))
        m, v = ref.r32(m), ref.r32(v)
    assert np.allclose(x, p.detach().numpy(), rtol=0, atol=5 * 1e-2 * 2.0 ** -22)


def test_checks_of_a_step_refuse_null_handles():
    lib, hp = ob.lib(), ob.adamw_hparams()
    assert lib.ob_adamw_check(None, None, None, None, None, None, ctypes.byref(hp), None) == ob._native.OB_ERR_ARG
    assert lib.ob_adamw8_check(None, None, None, None, None, None, None, None, ctypes.byref(hp), None) == ob._native.OB_ERR_ARG


def test_driver_refuses_a_bare_tensor():
    """It would be taken row by row."""
    with pytest.raises(TypeError, match="list"):
        ob.AdamW(torch.zeros(4, 4))


@pytest.mark.parametrize("key", ["betas", "eps", "bias_correction", "max_norm", "state_bits", "master", "rounding", "sr_seed",
                                 "grad_dtype", "amsgrad", "maximize"])
def test_driver_refuses_what_a_group_cannot_have(key):
    """Only the rate and the decay can differ between groups; another setting would be passed over."""
    with pytest.raises(ValueError, match=key):
        ob.AdamW([{"params": [torch.zeros(4)]}, {"params": [torch.zeros(4)], key: (7, 8) if key == "betas" else 7}])
    with pytest.raises(ValueError, match="GPU"):   # a name is none
        ob.AdamW([{"params": [torch.zeros(4)], "name": "a"}])
    own = {"amsgrad": False, "maximize": False, "betas": [0.8, 0.99]}
    with pytest.raises(ValueError, match="GPU"):   # nor is what all have
        ob.AdamW([{"params": [torch.zeros(4)], **own}], betas=(0.8, 0.99))
