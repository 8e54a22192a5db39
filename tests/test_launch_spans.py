"""What the training calls' launches are told to write, checked on the host
against the workspace they asked for (launch_spans_check.cpp: the library's
objects with a CUDA runtime that records launches)."""
import os
import subprocess

from dense_gemm_14_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")


def test_every_piece_writes_inside_the_workspace_and_over_nothing_else(tmp_path):
    build.build()
    exe = str(tmp_path / "launch_spans_check")
    objects = [os.path.join(build.BUILD_DIR, s.replace(".cu", ".o")) for s in build.SOURCES]
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", os.path.join(CUDA, "include"), "-I",
                    os.path.join(ROOT, "dense_gemm_14_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "launch_spans_check.cpp"), *objects, "-o", exe,
                    "-lpthread"], check=True, capture_output=True, text=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stdout)
