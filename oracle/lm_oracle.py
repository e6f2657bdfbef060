"""float64 definitions of the language-model operators (NumPy, per-step loops):
gated linear recurrence, gated feed-forward block, 8-bit checkpoints.  Written
from the formulas; shares no code with the library."""

import numpy as np

GROUP = 32


def sigmoid(x):
    x = np.asarray(x, np.float64)
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1 / (1 + e), e / (1 + e))


# ------------------------------------------------------------------- scan
def _coeffs(mode, p, q):
    """a, b and the candidate n of h' = a h + b."""
    if mode == "gated":
        n = np.tanh(q)
        return sigmoid(p), sigmoid(-p) * n, n
    return p, q, q


def scan_forward(mode, g, h0, lengths, dirs):
    """g [T, B, dirs*2*H] -> y [T, B, dirs*H], hy [dirs, B, H]."""
    T, B, W = g.shape
    H = W // (2 * dirs)
    g = np.asarray(g, np.float64).reshape(T, B, dirs, 2, H)
    y, hy = np.zeros((T, B, dirs, H)), np.zeros((dirs, B, H))
    for d in range(dirs):
        for b in range(B):
            n = T if lengths is None else min(max(int(lengths[b]), 0), T)
            h = np.zeros(H) if h0 is None else np.asarray(h0[d, b], np.float64)
            for t in (range(n) if d == 0 else range(n - 1, -1, -1)):
                a, add, _ = _coeffs(mode, g[t, b, d, 0], g[t, b, d, 1])
                h = a * h + add
                y[t, b, d] = h
            hy[d, b] = h
    return y.reshape(T, B, dirs * H), hy


def scan_backward(mode, g, h0, lengths, dy, dhy, dirs):
    """-> dg as g, dh0 [dirs, B, H]."""
    T, B, W = g.shape
    H = W // (2 * dirs)
    y, _ = scan_forward(mode, g, h0, lengths, dirs)
    y = y.reshape(T, B, dirs, H)
    g = np.asarray(g, np.float64).reshape(T, B, dirs, 2, H)
    dy = np.asarray(dy, np.float64).reshape(T, B, dirs, H)
    dg, dh0 = np.zeros(g.shape), np.zeros((dirs, B, H))
    for d in range(dirs):
        for b in range(B):
            n = T if lengths is None else min(max(int(lengths[b]), 0), T)
            walk = list(range(n) if d == 0 else range(n - 1, -1, -1))
            first = np.zeros(H) if h0 is None else np.asarray(h0[d, b], np.float64)
            dh = np.zeros(H) if dhy is None else np.asarray(dhy[d, b], np.float64)
            for i in range(len(walk) - 1, -1, -1):
                t = walk[i]
                before = y[walk[i - 1], b, d] if i else first
                p, q = g[t, b, d, 0], g[t, b, d, 1]
                a, _, cand = _coeffs(mode, p, q)
                dh = dh + dy[t, b, d]
                if mode == "gated":
                    dg[t, b, d, 0] = dh * (before - cand) * a * sigmoid(-p)
                    dg[t, b, d, 1] = dh * sigmoid(-p) * (1 - cand ** 2)
                else:
                    dg[t, b, d, 0], dg[t, b, d, 1] = dh * before, dh
                dh = dh * a
            dh0[d, b] = dh
    return dg.reshape(T, B, W), dh0


# -------------------------------------------------------------- checkpoint
def checkpoint_round(x):
    """x [rows, cols] as its 8-bit checkpoint holds it."""
    x = np.asarray(x, np.float64)
    out = np.empty_like(x)
    for c in range(0, x.shape[1], GROUP):
        v = x[:, c:c + GROUP]
        ok = np.isfinite(v).all(1, keepdims=True)
        v = np.where(ok, v, 0.0)
        top = np.abs(v).max(1, keepdims=True)
        e = np.maximum(np.frexp(np.where(top > 0, top, 2.0 ** -200))[1] - 7, -126)
        q = np.clip(np.rint(np.ldexp(v, -e)), -127, 127)
        out[:, c:c + GROUP] = np.where(ok, np.ldexp(q, e), np.nan)
    return out


# --------------------------------------------------------------------- ffn
def act_pair(act, g):
    """act(g) and its derivative."""
    if act == "gelu":
        c = np.sqrt(2 / np.pi)
        t = np.tanh(c * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    s = sigmoid(g)
    return (s, s * (1 - s)) if act == "sigmoid" else (g * s, s + g * s * (1 - s))


def ffn_forward(act, x, w_in, w_out):
    """-> y and the projections g, u."""
    F = w_out.shape[1]
    gu = x @ w_in.T
    g, u = gu[:, :F], gu[:, F:]
    return (act_pair(act, g)[0] * u) @ w_out.T, g, u


def ffn_backward(act, x, w_in, w_out, dy, save):
    """-> dx, dw_in, dw_out; save "int8": from the rounded x, g and u."""
    _, g, u = ffn_forward(act, x, w_in, w_out)
    if save == "int8":
        x, g, u = checkpoint_round(x), checkpoint_round(g), checkpoint_round(u)
    a, da = act_pair(act, g)
    dh = dy @ w_out
    dgu = np.concatenate([dh * u * da, dh * a], 1)
    return dgu @ w_in, dgu.T @ x, dy.T @ (a * u)
