"""CPU checks of ob_matmul: the host side's refusals and choices, and the binding's."""
import ctypes
import os
import subprocess

import pytest
import torch

import adam_ob_compress_amd as ob

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_host_side_of_products(tmp_path):
    exe = str(tmp_path / "product_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-D__HIP_PLATFORM_AMD__", "-I",
                    os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "adam_ob_compress_amd", "csrc"), "-I",
                    "/opt/rocm/include", os.path.join(ROOT, "tests", "product_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout


def test_layout_matches_the_header():
    # 4 extents, A and B with three strides each, C and D with two, two types, two factors, two flags, the workspace
    assert ctypes.sizeof(ob.ob_product) == 8 * (4 + 4 + 4 + 3 + 3) + 6 * 4 + 8
    assert ob.ob_product.d.offset == 8 * 15 and ob.ob_product.alpha.offset == 8 * 18 + 8


def test_refused_before_any_gpu_work():
    lib = ob.lib()
    assert lib.ob_matmul(None, None) == 1
    p = ob.ob_product(m=4, n=4, k=4, batch=1, in_type=1, alpha=1.0)
    assert lib.ob_matmul(ctypes.byref(p), None) == 1          # no pointers
    p.batch = 0
    assert lib.ob_matmul(ctypes.byref(p), None) == 0          # nothing to do
    p.in_type = 0
    assert lib.ob_matmul(ctypes.byref(p), None) == 3


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 4, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        ob.ob_matmul(x, x, x)
    with pytest.raises(TypeError, match="a must be"):
        ob.ob_matmul([1.0], x, x)
    with pytest.raises(TypeError):
        ob.ob_matmul(x, x, None)
