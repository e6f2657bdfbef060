"""The feed-forward block's backward pass where the values that RNN_SAVE_FULL keeps differ widely inside a group of
32 columns: one value far out, an infinity or a NaN must leave its neighbours as they are.

Tolerances: as in the block's own tests (derived there), with what is kept in bf16 mode counted value by value.  A kept
value is an fp16 number times a power of two that its group shares, which brings the group's largest finite magnitude
into [2^14, 2^15): half a step is 2^-11 of the value, and 2^-39 of the largest where the fp16 number is subnormal."""

import numpy as np
import pytest
import torch

from oracle import lm_oracle as O
from tests import test_gpu_lm_ffn as ffn

pytestmark = pytest.mark.gpu
U = ffn.U


def kept_error(v, dtype):
    if dtype == "f32":
        return np.zeros_like(v)
    pad = -v.shape[1] % 32
    top = np.abs(np.pad(v, ((0, 0), (0, pad)))).reshape(v.shape[0], -1, 32).max(2)
    return 2.0 ** -11 * np.abs(v) + 2.0 ** -39 * np.repeat(top, 32, 1)[:, :v.shape[1]]


def expected(c, act):
    """{name: (value, tolerance)} of the gradients of the weights, RNN_SAVE_FULL."""
    x, w_in, w_out, dy, F = c["x"], c["w_in"], c["w_out"], c["dy"], c["F"]
    half = ffn.HALF[c["dtype"]]
    gu = x @ w_in.T
    g, u = gu[:, :F], gu[:, F:]
    a, da = O.act_pair(act, g)
    p, h = u * da, a * u
    ea = 64 * U * (np.abs(a) + np.abs(g))
    eh = ea * np.abs(u) + half * np.abs(h)
    ea = ea + kept_error(a, c["dtype"])
    ep = 64 * U * (1 + np.abs(g)) * np.abs(u) + kept_error(p, c["dtype"])
    dh = dy @ w_out
    edh = c["D"] * U * (np.abs(dy) @ np.abs(w_out))
    dg, du = dh * p, dh * a
    edg = edh * (np.abs(p) + ep) + np.abs(dh) * ep
    edu = edh * (np.abs(a) + ea) + np.abs(dh) * ea
    edg, edu = edg + half * (np.abs(dg) + edg), edu + half * (np.abs(du) + edu)
    out = {}
    for k, left, el, right in (("dw_in", np.concatenate([dg, du], 1), np.concatenate([edg, edu], 1), x),
                               ("dw_out", h, eh, dy)):
        v = left.T @ right
        e = el.T @ np.abs(right) + c["M"] * U * ((np.abs(left) + el).T @ np.abs(right))
        out[k] = (v, e + half * (np.abs(v) + e))
    out["dw_out"] = tuple(v.T for v in out["dw_out"])
    return out


def with_outliers(M, D, F, dtype, bits):
    """One gate and one up column of every 32 are 2^bits times the others (a power of two: still exact)."""
    c = ffn.make(M, D, F, dtype, seed=5)
    c["w_in"][5:F:32] *= 2.0 ** bits
    c["w_in"][F + 9::32] *= 2.0 ** bits
    return c


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["sigmoid", "silu", "gelu"])
@pytest.mark.parametrize("size", [(40, 33, 70), (130, 64, 96), (300, 72, 321)], ids=lambda s: "x".join(map(str, s)))
def test_neighbours_of_large_values(dtype, act, size):
    print("CASE ffn outliers", dtype, act, size, flush=True)
    for bits in (6, 12):
        c = with_outliers(*size, dtype, bits)
        got, want = ffn.run(c, act, "full", ("dw_in", "dw_out")), expected(c, act)
        for k in ("dw_in", "dw_out"):
            x, (ref, tol) = got[k].double().cpu().numpy(), want[k]
            bad = np.abs(x - ref) > tol + 1e-30
            assert not bad.any(), (k, bits, int(bad.sum()), np.argwhere(bad)[:3].tolist())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("half", ["gate", "up"])
def test_infinities_and_nans_stay_in_their_column(dtype, value, half):
    """A weight that is no number: the gradients of the other columns' weights are what they are without it."""
    M, D, F, f = 200, 64, 100, 37
    c = ffn.make(M, D, F, dtype, seed=6)
    want = expected(c, "silu")
    c["w_in"][f if half == "gate" else F + f, 3] = value
    got = ffn.run(c, "silu", "full", ("dw_in", "dw_out"))
    others = np.arange(F) != f
    for k, rows in (("dw_in", np.concatenate([others, others])), ("dw_out", others)):
        x, (ref, tol) = got[k].double().cpu().numpy(), want[k]
        if k == "dw_out":
            x, ref, tol = x.T, ref.T, tol.T
        assert np.isfinite(x[rows]).all(), k
        assert (np.abs(x - ref)[rows] <= tol[rows] + 1e-30).all(), k
    assert not torch.isfinite(got["dw_out"][:, f]).any()
