"""CPU check of the largest matrices that a Muon plan takes: every load of its products stays within 32-bit offsets."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_reach_of_a_plans_tiles(tmp_path):
    exe = str(tmp_path / "muon_limits_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-D__HIP_PLATFORM_AMD__", "-I",
                    os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "adam_ob_compress_amd", "csrc"), "-I",
                    "/opt/rocm/include", os.path.join(ROOT, "tests", "muon_limits_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout
