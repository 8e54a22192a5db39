"""The training kernel's tile plan, checked on the host (train_plan_check.cpp)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")


def test_every_k_block_once_and_slots_within_the_workspace(tmp_path):
    exe = str(tmp_path / "train_plan_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", os.path.join(CUDA, "include"), "-I",
                    os.path.join(ROOT, "dense_gemm_14_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "train_plan_check.cpp"), "-o", exe],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, (r.returncode, r.stdout)
