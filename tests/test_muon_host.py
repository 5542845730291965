"""CPU checks of the Muon step, the norms and clipping: the host side's plans and refusals, and the binding's."""
import ctypes
import os
import subprocess

import pytest
import torch

import adam_ob_compress_amd as ob

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_host_side_of_plans(tmp_path):
    exe = str(tmp_path / "muon_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-D__HIP_PLATFORM_AMD__", "-I",
                    os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "adam_ob_compress_amd", "csrc"), "-I",
                    "/opt/rocm/include", os.path.join(ROOT, "tests", "muon_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout


def test_layout_matches_the_header():
    assert ctypes.sizeof(ob.ob_muon_hparams) == 32 and ob.ob_muon_hparams.nesterov.offset == 16


def test_null_handles_are_refused():
    lib = ob.lib()
    P = ctypes.c_void_p
    hp = ob.muon_hparams()
    h = P(1)
    assert lib.ob_muon_create(None, None, None, ctypes.byref(h)) == 1 and h.value is None
    assert lib.ob_muon_create(None, None, None, None) == 1
    assert lib.ob_muon_destroy(None) == 1 and lib.ob_muon_workspace(None) == -1
    assert lib.ob_muon_step(None, None, None, None, None, None, ctypes.byref(hp), None, None) == 1
    assert lib.ob_muon_check(None, None, None, None, None, None, ctypes.byref(hp), None) == 1
    assert lib.ob_tensor_norms_workspace(None) == -1
    assert lib.ob_tensor_norms(None, None, 1.0, 0, P(0x1000), P(0x2000), None) == 1
    assert lib.ob_clip_grads(None, None, None, P(0x1000), 1.0, 1.0, 0, None) == 1


def test_binding_refuses_host_tensors():
    x = torch.zeros(8, 8)
    with pytest.raises(ValueError, match="GPU"):
        ob.Muon([x])
    with pytest.raises(ValueError, match="GPU"):
        ob.GradClip([x], max_norm=1.0)
    with pytest.raises(ValueError, match="no matrix"):
        ob.Muon([torch.zeros(8)])
    with pytest.raises(ValueError, match="twice"):
        ob.Muon([x, x])
    with pytest.raises(ValueError, match="twice"):
        ob.GradClip([x, x], max_norm=1.0)
    with pytest.raises(ValueError, match="norm must be"):
        ob.GradClip([x], max_norm=1.0, norm="1")
    with pytest.raises(ValueError, match="own momentum"):
        ob.Muon([{"params": x, "momentum": 0.5}])
    with pytest.raises(TypeError, match="list"):
        ob.GradClip(x, max_norm=1.0)
