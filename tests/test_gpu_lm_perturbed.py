"""Race detection for the scan's exchange: the perturbed build (-DRNN_PERTURB) pauses pseudo-randomly before a chunk is
taken, before it is published and before a state is passed on, so that chunks meet in orders that the normal build
hardly ever has.  Every output and gradient has to be bitwise the normal build's."""

import os
import subprocess
import sys

import numpy as np
import pytest

from layer_rnn_forward_amd.build import PERTURB_LIB
from tests import lm_perturb_cases

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.timeout(300)
def test_perturbed_scan_is_bitwise_equal(tmp_path):
    assert os.path.exists(PERTURB_LIB), "the perturbed test build is missing (run build())"
    ref, out = lm_perturb_cases.run_all(), tmp_path / "perturbed.npz"
    r = subprocess.run([sys.executable, "-u", os.path.join(ROOT, "tests", "lm_perturb_cases.py"), str(out)],
                       env=dict(os.environ, RNN_LIB=PERTURB_LIB), cwd=ROOT, capture_output=True, text=True, timeout=240)
    print(r.stdout[-2000:], r.stderr[-2000:], flush=True)
    assert r.returncode == 0 and "perturb" in r.stdout.splitlines()[0]
    got = np.load(out)
    assert sorted(got.files) == sorted(ref)
    for k, v in ref.items():
        assert np.isfinite(v).all() and np.array_equal(got[k].view(np.uint32), v.view(np.uint32)), k
