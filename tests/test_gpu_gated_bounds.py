"""The gated block and clipping in the debug-bounds build: the same bits as the default build, and no failed
index check (tests/gated_bounds_run.py in separate processes)."""
import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _run(variant, out):
    proc = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "gated_bounds_run.py"), out],
                          env=dict(os.environ, OWQ_LIB_VARIANT=variant), capture_output=True, text=True, timeout=600)
    assert proc.returncode == 0, proc.stdout[-2000:] + proc.stderr[-4000:]
    return np.load(out)


def test_debug_bounds_build_matches_and_reports_nothing(tmp_path):
    from weight_only_mixed_owq_b200 import build as b
    if not b.up_to_date(b.LIB_BOUNDS):
        b.build(debug_bounds=True)
    ref, dbg = _run("", str(tmp_path / "default.npz")), _run("bounds", str(tmp_path / "bounds.npz"))
    assert str(dbg["version"]).endswith("+debug-bounds") and sorted(ref.files) == sorted(dbg.files)
    compared = 0
    for key in ref.files:
        if key == "version":
            continue
        if key.endswith("_status"):
            assert int(ref[key]) == 0 and int(dbg[key]) == 0, key
            continue
        p, q = ref[key], dbg[key]
        assert p.shape == q.shape and p.dtype == q.dtype and np.array_equal(p.view(np.uint8), q.view(np.uint8)), key
        compared += 1
    assert compared >= 100
