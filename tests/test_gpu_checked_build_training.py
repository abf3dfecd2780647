"""The access-checking build of head norms with the rotation, token log probabilities
and AdamW: ragged, unaligned and padded workloads in a child process.  No access may
be reported, and every result must equal the release library's bytes."""
import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.slow
def test_checked_build_reports_nothing_and_matches_release(rp, tmp_path):
    from verifiable_repops_gemm_gb300 import build
    lib = build.build(checked=True)
    out = tmp_path / "checked.npz"
    r = subprocess.run([sys.executable, os.path.join(HERE, "checked_build_training_run.py"), lib, str(out)],
                       capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    import checked_build_training_run
    want = checked_build_training_run.workloads(rp)
    got = np.load(out)
    assert sorted(got.files) == sorted(want) and len(want) > 500
    for name, w in want.items():
        assert np.array_equal(got[name], w), name
