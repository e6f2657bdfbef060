"""Without its compiled entries the package loads, and the operators' checks and queries are the same; no GPU."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import sys, warnings
sys.modules["layer_rnn_forward_amd._call"] = None        # its import fails
import torch
import layer_rnn_forward_amd as R
warnings.simplefilter("error")
h = R.rnn_create("lstm", 1, 1, 16, 64, "f32")            # the recurrent layers do not need them: no warning either
assert R.rnn_workspace_size(h, 5, 4, 0) > 0
assert R.rnn_scan_workspace_size(10, 2, 8) > 0
warnings.simplefilter("always")
with warnings.catch_warnings(record=True) as said:
    assert R.rnn_checkpoint_size(3, 33) == 105
    assert R.rnn_checkpoint_size(1, 32) == 33
    for call in (lambda: R.rnn_scan_step("gated", torch.zeros(2, 7), None, None, torch.zeros(2, 3)),
                 lambda: R.rnn_ffn_forward("relu", *[torch.zeros(4, 8)] * 5),
                 lambda: R.rnn_checkpoint_load(torch.zeros(64), torch.zeros(4, 8))):
        try:
            call()
        except ValueError:
            continue
        raise AssertionError("not refused")
assert len(said) == 1 and "_call.so" in str(said[0].message), said
print("fine")
"""


def test_package_without_compiled_entries():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split()[-1] == "fine", r.stderr
