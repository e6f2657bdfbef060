"""Scans for the ordering-perturbation test: ``python tests/lm_perturb_cases.py OUT.npz`` with ``RNN_LIB`` set to the
build to run."""

import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

CASES = [("gated", "bf16", 3000, 2, 200, 2, [3000, 1700]), ("gated", "f32", 1500, 5, 75, 1, None),
         ("linear", "bf16", 5000, 1, 1000, 1, None), ("linear", "f32", 700, 3, 130, 2, [700, 0, 64])]


def run_all():
    from tests import test_gpu_lm_scan as scan
    out = {}
    for i, (mode, dtype, T, B, H, dirs, lengths) in enumerate(CASES):
        print("case", i, flush=True)
        got = scan.run(scan.make(mode, dtype, T, B, H, dirs, lengths, seed=9))
        out |= {f"{i}.{k}": v.float().cpu().numpy() for k, v in got.items()}
    return out


if __name__ == "__main__":
    import layer_rnn_forward_amd as R
    print("library", R.lib_path(), flush=True)
    np.savez(sys.argv[1], **run_all())
