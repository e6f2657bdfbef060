"""The oracle of the state-space block's operators: its gradients against differences of its values and against
torch's in float64, and its bounds against an evaluation in float32."""

import numpy as np
import pytest
import torch

from oracle import block_oracle as O
from oracle.bounds import Bound


def rand(seed, *shape):
    return np.random.default_rng(seed).normal(size=shape)


def differences(f, args, name, seed, step=1e-6):
    """(directional difference, direction) of the scalar f at args[name]."""
    d = rand(seed, *args[name].shape)
    up, down = dict(args), dict(args)
    up[name], down[name] = args[name] + step * d, args[name] - step * d
    return (f(up) - f(down)) / (2 * step), d


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm(kind):
    M, D = 5, 7
    a = {"s": rand(1, M, D), "w": rand(2, D), "b": rand(3, D)}
    dy = rand(4, M, D)

    def f(v):
        return (O.norm_forward(kind, v["s"], v["w"], v["b"], 1e-3)[0].v * dy).sum()

    dx, dw, db = O.norm_backward(kind, a["s"], a["w"], 1e-3, dy, None)
    for name, g in (("s", dx), ("w", dw), ("b", db)):
        want, d = differences(f, a, name, 9)
        assert abs((g.v * d).sum() - want) <= 1e-7 * max(1, abs(want)), name
    if kind == "layer":
        y = torch.nn.functional.layer_norm(torch.tensor(a["s"]), (D,), torch.tensor(a["w"]), torch.tensor(a["b"]), 1e-3)
        assert np.allclose(y.numpy(), O.norm_forward(kind, a["s"], a["w"], a["b"], 1e-3)[0].v, rtol=1e-12)


@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("T,K,lengths", [(6, 4, None), (5, 3, [5, 0, 1]), (2, 4, [2, 1, 0]), (0, 3, None), (4, 1, [1, 4, 0])])
def test_conv(act, T, K, lengths):
    B, C = 3, 4
    a = {"x": rand(1, T, B, C), "w": rand(2, C, K), "bias": rand(3, C), "s0": rand(4, K - 1, B, C)}
    dy, dsy = rand(5, T, B, C), rand(6, K - 1, B, C)

    def f(v):
        r = O.conv(act, v["x"], v["w"], v["bias"], v["s0"], lengths)
        return (r["y"].v * dy).sum() + (r["sy"].v * dsy).sum()

    r = O.conv(act, a["x"], a["w"], a["bias"], a["s0"], lengths, dy, dsy)
    for name in a:
        want, d = differences(f, a, name, 9)
        assert abs((r["d" + name].v * d).sum() - want) <= 1e-7 * max(1, abs(want)), name
    if lengths is None and T:
        xs = torch.tensor(np.concatenate([a["s0"], a["x"]])).permute(1, 2, 0)
        v = torch.nn.functional.conv1d(xs, torch.tensor(a["w"])[:, None], torch.tensor(a["bias"]), groups=C).permute(2, 0, 1)
        v = torch.nn.functional.silu(v) if act == "silu" else v
        assert np.allclose(v.numpy(), r["y"].v, rtol=1e-12, atol=1e-14)


@pytest.mark.parametrize("mode", ["softplus", "linear"])
@pytest.mark.parametrize("T,G,lengths,gated", [(5, 1, None, True), (6, 2, [6, 0, 3], True), (4, 2, [0, 4, 1], False), (0, 1, None, True)])
def test_ssm(mode, T, G, lengths, gated):
    B, E, N = 3, 4, 3
    a = {"u": rand(1, T, B, E), "delta": rand(2, T, B, E), "A": -np.abs(rand(3, E, N)), "Bm": rand(4, T, B, G * N),
         "Cm": rand(5, T, B, G * N), "D": rand(6, E), "z": rand(7, T, B, E), "delta_bias": rand(8, E), "h0": rand(9, B, E, N)}
    if not gated:
        a["z"] = None
    if mode == "linear":                 # negative d let states grow until a difference of values has no digits left
        a["delta"], a["delta_bias"] = np.abs(a["delta"]), np.abs(a["delta_bias"])
    dy, dhy = rand(10, T, B, E), rand(11, B, E, N)
    order = ("u", "delta", "A", "Bm", "Cm", "D", "z", "delta_bias", "h0")

    def f(v):
        r = O.ssm(mode, *(v[k] for k in order), lengths)
        return (r["y"].v * dy).sum() + (r["hy"].v * dhy).sum()

    r = O.ssm(mode, *(a[k] for k in order), lengths, dy, dhy)
    for name in order:
        if a[name] is None:
            assert "d" + name not in r
            continue
        want, d = differences(f, a, name, 12)
        assert abs((r["d" + name].v * d).sum() - want) <= 2e-7 * max(1, abs(want)), name


def test_ssm_by_hand():
    """One channel, two states, two steps: d = 1 and 2, a = 1/2 and 1 (A = -ln 2 and 0)."""
    A = np.array([[-np.log(2.0), 0.0]])
    one = np.ones((2, 1, 1))
    r = O.ssm("linear", one * [[[3.0]], [[1.0]]], one * [[[1.0]], [[2.0]]], A, one * [1.0, 2.0], one * [1.0, 1.0],
              np.array([10.0]), None, None, np.full((1, 1, 2), 4.0), None)
    # h1 = (4/2 + 3, 4 + 6) = (5, 10); h2 = (5/4 + 2, 10 + 4) = (3.25, 14)
    assert np.allclose(r["hy"].v, [[[3.25, 14.0]]])
    assert np.allclose(r["y"].v.ravel(), [15 + 30, 17.25 + 10])


def test_bounds_hold_in_float32():
    """The same operations in numpy's float32 stay within the bounds."""
    rng = np.random.default_rng(0)
    x, y = rng.normal(size=(2, 4000)).astype(np.float32)
    f = np.float32

    def exp(v):                          # as the kernels: base 2, right to 1 unit in the last place (numpy's own is not)
        return np.exp2((v * f(np.log2(np.e))).astype(np.float64)).astype(f)

    for got, want in (((x * y) + x, Bound(x) * y + x), (exp(x), Bound(x).exp()), ((x * y).reshape(40, 100).sum(1), (Bound(x) * y).reshape(40, 100).sum(1)),
                      (f(1) / (f(1) + exp(-x)), Bound(x).sigmoid()), (f(1) / np.sqrt(x * x + f(1)), (Bound(x) * x + 1.0).rsqrt()),
                      (np.maximum(x, f(0)) + np.log1p(exp(-np.abs(x))), Bound(x).softplus())):
        assert got.dtype == np.float32 and (np.abs(got - want.v) <= want.e).all()
