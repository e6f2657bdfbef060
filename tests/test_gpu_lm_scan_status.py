"""The scan's expired waits: which call notes and clears them, and that a step's host sees them."""

import os
import subprocess
import sys

import pytest
import torch

import layer_rnn_forward_amd as R
from tests import test_gpu_lm_scan as scan

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def calls(T, B=2, H=64):
    c = scan.make("gated", "bf16", T, B, H, 1)
    g, h0, dy, dhy = (c[k].cuda() for k in ("g", "h0", "dy", "dhy"))
    y, hy, dg, dh0 = torch.empty_like(dy), torch.empty_like(h0), torch.empty_like(g), torch.empty_like(h0)
    ws = torch.full((R.rnn_scan_workspace_size(T, B, H, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    return (ws, lambda: R.rnn_scan_forward("gated", g, h0, None, y, hy, ws),
            lambda: R.rnn_scan_backward("gated", g, h0, None, dy, dhy, dg, dh0, ws))


@pytest.mark.parametrize("T", [0, 20, 3000])   # no step, one chunk, many
def test_words(T):
    ws, forward, backward = calls(T)
    words = ws[:8].view(torch.int32)
    forward()
    assert words.tolist() == [0, 0] and R.rnn_scan_status(ws) == 0
    backward()
    assert words.tolist() == [0, 0] and R.rnn_scan_status(ws) == 0
    words.copy_(torch.tensor([1, 0], dtype=torch.int32))     # as a forward wait that expired would leave them
    assert R.rnn_scan_status(ws) == -7
    backward()
    assert words.tolist() == [1, 0] and R.rnn_scan_status(ws) == -7
    words.copy_(torch.tensor([0, 1], dtype=torch.int32))     # as a backward wait would
    assert R.rnn_scan_status(ws) == -7
    backward()
    assert R.rnn_scan_status(ws) == 0
    words.fill_(1)
    forward()
    assert words.tolist() == [0, 0] and R.rnn_scan_status(ws) == 0


def test_forced_timeout_is_reported():
    """A limit of 0 from the host: every wait whose words are not there expires at once, every workgroup ends."""
    code = ("from tests import test_gpu_lm_scan_status as t\n"
            "import layer_rnn_forward_amd as R\n"
            "ws, forward, backward = t.calls(20000)\n"
            "forward()\n"
            "print('STATUS', R.rnn_scan_status(ws))\n"
            "backward()\n"
            "print('STATUS', R.rnn_scan_status(ws))\n")
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, RNN_SPIN_LIMIT="0"), capture_output=True, text=True,
                       timeout=100, cwd=ROOT)
    assert r.returncode == 0, r.stderr
    assert r.stdout.count("STATUS -7") == 2, r.stdout


def test_refusals():
    with pytest.raises(R.RNNError):
        R.rnn_scan_status(torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="device"):
        R.rnn_scan_status(torch.zeros(512, dtype=torch.uint8))
