"""Gradients of the scan's gates where the candidate's tangent is all but 1: relative to themselves."""

import numpy as np
import pytest
import torch

from oracle import lm_oracle as O
from tests import test_gpu_lm_scan as scan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slopes_of_saturated_candidates(dtype):
    """dq = dh s(-p) (1 - tanh^2 q): relative to itself, however near the tangent is to 1 (fp32: 64 roundings of the
    value, for the exponential's argument 2 |q| log2(e) roundings more; bf16: half a step on top)."""
    q = torch.tensor([0.0, 0.01, 0.06, 0.07, 0.5, 1.0, 2.0, 4.0, 6.0, 8.0, 8.5, 9.0, 10.0, 15.0, 20.0, 30.0])
    q = torch.cat([q, -q])
    H = q.numel()
    for T in (1, 150):
        g = torch.zeros(T, 1, 2 * H)
        g[:, :, H:] = q
        c = dict(mode="gated", dtype=dtype, T=T, B=1, H=H, dirs=1, lengths=None, g=g.to(scan.DT[dtype]),
                 dy=torch.ones(T, 1, H).to(scan.DT[dtype]), h0=None, dhy=None)
        dq = scan.run(c)["dg"][:, :, H:].double().cpu().numpy()
        # with p = 0 the gradient that reaches a step does not depend on q; 1 - tanh^2 q is 4 t / (1 + t)^2 with
        # t = e^(-2 |q|), which loses no digits
        zero, one = np.zeros((T, 1, 2 * H)), np.ones((T, 1, H))
        dh = 2 * O.scan_backward("gated", zero, None, None, one, None, 1)[0][:, :, H:]
        x = c["g"].double().numpy()[:, :, H:]
        t = np.exp(-2 * np.abs(x))
        ref = dh * 0.5 * 4 * t / (1 + t) ** 2
        tol = (64 + 2 * np.abs(x) * 1.45) * scan.U * ref
        tol = tol + scan.HALF[dtype] * (ref + tol) + 2.0 ** -126
        assert (np.abs(dq - ref) <= tol).all(), (T, dtype, (np.abs(dq - ref) / tol).max())
