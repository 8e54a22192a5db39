"""The training products on the build with device-side bounds checks: every
store of a tile, of a split tile's sums and of a tile's statistics is tested
against its buffer; none may fail, and the results are the product build's."""
import os
import subprocess
import sys

import numpy as np
import pytest

from dense_gemm_14_gb300 import build

import training_checks_worker as worker

pytestmark = pytest.mark.gpu


def test_checked_build_agrees_and_reports_nothing(tmp_path):
    lib = build.build(checked=True)
    out = tmp_path / "checked.npz"
    r = subprocess.run([sys.executable, worker.__file__, str(out)], capture_output=True, text=True,
                       timeout=900, env=dict(os.environ, GEMM14_LIB=lib))
    assert r.returncode == 0, r.stderr[-3000:]
    got = np.load(out)
    assert str(got["lib"]) == lib and int(got["status"]) == 0
    want, status = worker.run_all()
    assert status == 0
    for i, a in enumerate(want):
        assert np.array_equal(got[f"a{i}"], a, equal_nan=True), i
