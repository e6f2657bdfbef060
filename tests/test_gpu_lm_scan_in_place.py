"""A scan's last state written over its first one (hy the same tensor as h0, dh0 as dhy): bitwise the results of
separate tensors, also where the workgroups meet in other orders (the build with perturbed ordering points)."""

import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import layer_rnn_forward_amd as R  # noqa: E402
from tests import test_gpu_lm_scan as scan  # noqa: E402

pytestmark = pytest.mark.gpu

# T, B, H, dirs, lengths: one chunk, one group of chunks, the last chunk in the first group, many groups
SIZES = [(40, 2, 64, 1, None), (300, 3, 70, 2, [300, 0, 11]), (1024, 1, 512, 1, None), (3000, 2, 130, 2, None)]


def compare(mode, dtype, T, B, H, dirs, lengths):
    c = scan.make(mode, dtype, T, B, H, dirs, lengths, seed=12)
    want = scan.run(c)
    g, n, dy = (scan.cuda(c[k]) for k in ("g", "lengths", "dy"))
    ws = torch.full((R.rnn_scan_workspace_size(T, B, H, dirs),), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        h, d = c["h0"].cuda(), c["dhy"].cuda()
        y, dg = torch.empty_like(want["y"]), torch.empty_like(want["dg"])
        R.rnn_scan_forward(mode, g, h, n, y, h, ws)
        R.rnn_scan_backward(mode, g, h, n, dy, d, dg, d, ws)
        for k, v in (("y", y), ("hy", h), ("dg", dg), ("dh0", d)):
            assert torch.equal(v, want[k]), k


@pytest.mark.parametrize("mode,dtype", [("gated", "bf16"), ("linear", "f32")])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s[:4])))
def test_last_state_over_the_first(mode, dtype, size):
    print("CASE scan in place", mode, dtype, size, flush=True)
    compare(mode, dtype, *size)


def test_pieces_carry_their_state():
    """A sequence in pieces, each from the state that the piece before left in the same tensor."""
    c = scan.make("gated", "f32", 900, 2, 50, 1)
    want = scan.expected(c)
    g, h = c["g"].cuda(), c["h0"].cuda()
    y = torch.empty(900, 2, 50, device="cuda")
    for a, b in ((0, 500), (500, 501), (501, 900)):
        ws = torch.empty(R.rnn_scan_workspace_size(b - a, 2, 50, 1), dtype=torch.uint8, device="cuda")
        R.rnn_scan_forward("gated", g[a:b], h, None, y[a:b], h, ws)
    scan.check({"y": y, "hy": h}, want)


@pytest.mark.timeout(300)
def test_perturbed_order():
    from layer_rnn_forward_amd.build import PERTURB_LIB
    assert os.path.exists(PERTURB_LIB), "the perturbed test build is missing (run build())"
    r = subprocess.run([sys.executable, "-u", os.path.abspath(__file__)], env=dict(os.environ, RNN_LIB=PERTURB_LIB), cwd=ROOT,
                       capture_output=True, text=True, timeout=240)
    print(r.stdout[-2000:], r.stderr[-2000:], flush=True)
    assert r.returncode == 0 and "perturb" in r.stdout.splitlines()[0] and r.stdout.splitlines()[-1] == "same"


if __name__ == "__main__":
    print("library", R.lib_path(), flush=True)
    for size in SIZES:
        for case in (("gated", "bf16"), ("linear", "f32")):
            print("case", case, size, flush=True)
            compare(*case, *size)
    print("same", flush=True)
