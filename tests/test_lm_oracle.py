"""The language-model operators' oracle: gradients against central differences
of its own forward pass, the checkpoint's grid, and hand-worked values."""

import numpy as np
import pytest

from oracle import lm_oracle as O


@pytest.mark.parametrize("mode", ["gated", "linear"])
@pytest.mark.parametrize("dirs", [1, 2])
@pytest.mark.parametrize("ragged", [False, True])
def test_scan_gradients(mode, dirs, ragged):
    rng = np.random.default_rng(3)
    T, B, H = 5, 3, 2
    g = rng.normal(size=(T, B, dirs * 2 * H))
    h0, dy, dhy = rng.normal(size=(dirs, B, H)), rng.normal(size=(T, B, dirs * H)), rng.normal(size=(dirs, B, H))
    lengths = [5, 0, 3] if ragged else None

    def loss(g, h0):
        y, hy = O.scan_forward(mode, g, h0, lengths, dirs)
        return (y * dy).sum() + (hy * dhy).sum()

    dg, dh0 = O.scan_backward(mode, g, h0, lengths, dy, dhy, dirs)
    for x, grad in ((g, dg), (h0, dh0)):
        for i in np.ndindex(*x.shape):
            e = np.zeros(x.shape)
            e[i] = 1e-5
            f = (loss(x + e, h0) - loss(x - e, h0)) if x is g else (loss(g, x + e) - loss(g, x - e))
            assert abs(f / 2e-5 - grad[i]) < 1e-8, i


def test_scan_by_hand():
    # a = 1/2 twice, b = 1: h = 1, 3/2; the second direction walks back: h = 1 + 1/2 h
    g = np.array([[[0.5, 1.0, 0.5, 1.0]], [[0.5, 1.0, 0.5, 1.0]]])
    y, hy = O.scan_forward("linear", g, None, None, 2)
    assert y.tolist() == [[[1.0, 1.5]], [[1.5, 1.0]]] and hy.ravel().tolist() == [1.5, 1.5]


@pytest.mark.parametrize("act", ["sigmoid", "silu", "gelu"])
def test_ffn_gradients(act):
    rng = np.random.default_rng(4)
    M, D, F = 3, 4, 5
    ops = [rng.normal(size=s) for s in ((M, D), (2 * F, D), (D, F))]
    dy = rng.normal(size=(M, D))
    grads = O.ffn_backward(act, *ops, dy, "full")
    for k in range(3):
        for i in np.ndindex(*ops[k].shape):
            up, dn = [o.copy() for o in ops], [o.copy() for o in ops]
            up[k][i] += 1e-5
            dn[k][i] -= 1e-5
            f = ((O.ffn_forward(act, *up)[0] - O.ffn_forward(act, *dn)[0]) * dy).sum() / 2e-5
            assert abs(f - grads[k][i]) < 1e-7, (k, i)


def test_checkpoint_grid():
    x = np.array([[1.0, 127.0, -128.0, 0.5, 1.5, 2.5]])
    # the largest magnitude, 128, is 2^7: units of 2
    assert O.checkpoint_round(x).tolist() == [[0.0, 128.0, -128.0, 0.0, 2.0, 2.0]]
    assert O.checkpoint_round(np.array([[127.0, 0.5, 1.5, 127.6]])).tolist() == [[127.0, 0.0, 2.0, 127.0]]
    assert (O.checkpoint_round(np.zeros((2, 40))) == 0).all()
    bad = O.checkpoint_round(np.array([[1.0] * 32 + [2.0, np.inf]]))
    assert (bad[0, :32] == 1.0).all() and np.isnan(bad[0, 32:]).all()
    rng = np.random.default_rng(5)
    x = rng.normal(size=(9, 77)) * np.exp(rng.normal(size=(9, 1)) * 20)
    back = O.checkpoint_round(x)
    assert (O.checkpoint_round(back) == back).all()          # on the grid already
    for c in range(0, 77, 32):
        top = np.abs(x[:, c:c + 32]).max(1, keepdims=True)
        assert (np.abs(back - x)[:, c:c + 32] <= top / 64 * 0.5 + top / 128).all()
