"""The operators of a state-space block in 64 bits, step by step from their formulas, with bounds on what fp32 may lose
(oracle/bounds.py): normalisation, causal convolution, selective state-space scan.

Inputs are numpy arrays (as the element type holds them); results are ``Bound`` values."""

import numpy as np

from .bounds import Bound, stack


# -------------------------------------------------------------------- norm
def norm_forward(kind, s, weight, bias, eps):
    """y, (m, rstd) of rows s [M, D]."""
    D = s.shape[1]
    s = Bound(s)
    m = s.sum(1) * (1.0 / D) if kind == "layer" else Bound(np.zeros(s.v.shape[0]))
    c = s - m.reshape(-1, 1)
    rstd = ((c * c).sum(1) * (1.0 / D) + eps).rsqrt()
    y = c * rstd.reshape(-1, 1)
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, m, rstd


def norm_backward(kind, s, weight, eps, dy, dtotal):
    """dx, dweight, dbias."""
    D = s.shape[1]
    _, m, rstd = norm_forward(kind, s, None, None, eps)
    xh = (Bound(s) - m.reshape(-1, 1)) * rstd.reshape(-1, 1)
    dy = Bound(dy)
    g = dy * weight if weight is not None else dy
    dx = g - xh * ((g * xh).sum(1) * (1.0 / D)).reshape(-1, 1)
    if kind == "layer":
        dx = dx - (g.sum(1) * (1.0 / D)).reshape(-1, 1)
    dx = dx * rstd.reshape(-1, 1)
    if dtotal is not None:
        dx = dx + dtotal
    return dx, (dy * xh).sum(0), dy.sum(0)


# -------------------------------------------------------------------- conv
def _silu(v):
    s = v.sigmoid()
    return v * s, s * (1.0 + v * (1.0 - s))


def conv(act, x, w, bias, s0, lengths, dy=None, dsy=None):
    """y, sy and, with dy, dx, dw, dbias, ds0 for x [T, B, C]."""
    T, B, C = x.shape
    K = w.shape[1]
    if s0 is None:
        s0 = np.zeros((K - 1, B, C))
    n = [T] * B if lengths is None else [min(max(int(m), 0), T) for m in lengths]
    live = np.arange(T)[:, None] < np.asarray(n)[None]
    x = np.where(live[:, :, None], x, 0.0)
    xs = np.concatenate([s0, x])
    y, slope = [], []
    for t in range(T):
        v = Bound(np.zeros((B, C)) + (0.0 if bias is None else bias))
        for k in range(K):
            v = v + Bound(xs[t + k]) * w[:, k]
        f, d = _silu(v) if act == "silu" else (v, Bound(np.ones((B, C))))
        y.append(f.where(live[t][:, None]))
        slope.append(d)
    sy = np.stack([xs[n[b]:n[b] + K - 1, b] for b in range(B)], 1)
    out = {"y": stack(y) if T else Bound(np.zeros((T, B, C))), "sy": Bound(sy)}
    if dy is None:
        return out
    dxs = [Bound(np.zeros((B, C))) for _ in range(T + K - 1)]
    dw, db = [], []
    for t in range(T):
        dv = (Bound(np.where(live[t][:, None], dy[t], 0.0)) * slope[t]).where(live[t][:, None])
        for k in range(K):
            dxs[t + k] = dxs[t + k] + dv * w[:, k]
        dw.append(stack([dv * xs[t + k] for k in range(K)]))
        db.append(dv)
    if dsy is not None:
        for b in range(B):
            for j in range(K - 1):
                at = dxs[n[b] + j]
                v, e = at.v.copy(), at.e.copy()
                more = at + dsy[j]
                v[b], e[b] = more.v[b], more.e[b]
                dxs[n[b] + j] = Bound(v, e)
    zero = Bound(np.zeros((1, K, B, C)))
    out["dw"] = (stack(dw) if T else zero).sum((0, 2))
    out["dw"] = Bound(out["dw"].v.T, out["dw"].e.T)
    out["dbias"] = (stack(db) if T else Bound(np.zeros((1, B, C)))).sum((0, 1))
    every = stack(dxs) if dxs else Bound(np.zeros((0, B, C)))
    out["ds0"], out["dx"] = every[:K - 1], every[K - 1:]
    return out


# --------------------------------------------------------------------- ssm
def ssm(mode, u, delta, A, Bm, Cm, D, z, delta_bias, h0, lengths, dy=None, dhy=None):
    """y, hy and, with dy, every gradient; u, delta, z [T, B, E], Bm, Cm [T, B, G * N], A [E, N]."""
    T, B, E = u.shape
    N = A.shape[1]
    G = Bm.shape[2] // N
    n = np.asarray([T] * B if lengths is None else [min(max(int(m), 0), T) for m in lengths])

    def states(v):                       # [B, G N] -> [B, E, N]
        return np.repeat(v.reshape(B, G, N), E // G, 1)

    h = Bound(np.zeros((B, E, N)) if h0 is None else h0)
    kept, ys = [], []
    for t in range(T):
        on = (t < n)[:, None]
        on3 = on[:, :, None]
        ut, zt = np.where(on, u[t], 0.0), np.where(on, z[t], 0.0) if z is not None else None
        Bt, Ct = np.where(on3, states(Bm[t]), 0.0), np.where(on3, states(Cm[t]), 0.0)
        pre = Bound(np.where(on, delta[t], 0.0)) + (0.0 if delta_bias is None else delta_bias)
        d = (pre.softplus() if mode == "softplus" else pre).where(on)
        du = d * ut
        a = (d.reshape(B, E, 1) * A).exp()
        before = h
        h = (a * h + du.reshape(B, E, 1) * Bt)
        h = Bound(np.where(on3, h.v, before.v), np.where(on3, h.e, before.e))
        o = (h * Ct).sum(2)
        if D is not None:
            o = o + Bound(ut) * D
        y = o
        if z is not None:
            y = o * _silu(Bound(zt))[0]
        ys.append(y.where(on))
        kept.append((ut, zt, Bt, Ct, pre, d, du, a, before, h, o, on))
    out = {"y": stack(ys) if T else Bound(np.zeros((T, B, E))), "hy": h}
    if dy is None:
        return out
    g = Bound(np.zeros((B, E, N)) if dhy is None else dhy)
    rows = {k: [] for k in ("du", "ddelta", "dz", "dBm", "dCm", "dA", "dD")}
    for t in range(T - 1, -1, -1):
        ut, zt, Bt, Ct, pre, d, du, a, before, after, o, on = kept[t]
        do = Bound(np.where(on, dy[t], 0.0))
        if z is not None:
            f, slope = _silu(Bound(zt))
            rows["dz"].append((do * o * slope).where(on))
            do = do * f
        do3, on3 = do.reshape(B, E, 1), on[:, :, None]
        rows["dCm"].append((do3 * after).where(on3).reshape(B, G, E // G, N).sum(2).reshape(B, G * N))
        later = g
        g = g + do3 * Ct
        rows["dBm"].append((g * du.reshape(B, E, 1)).where(on3).reshape(B, G, E // G, N).sum(2).reshape(B, G * N))
        gb = (g * Bt).sum(2)
        rows["du"].append((d * gb + (do * D if D is not None else 0.0)).where(on))
        rows["dD"].append((do * ut).where(on))
        x = g * a * before
        rows["dA"].append((x * d.reshape(B, E, 1)).where(on3))
        dd = (x * A).sum(2) + gb * ut
        if mode == "softplus":
            dd = dd * pre.sigmoid()
        rows["ddelta"].append(dd.where(on))
        g = g * a
        g = Bound(np.where(on3, g.v, later.v), np.where(on3, g.e, later.e))
    for k in ("du", "ddelta", "dz", "dBm", "dCm"):
        if rows[k]:
            out[k] = stack(rows[k][::-1])
        elif k != "dz" or z is not None:
            out[k] = Bound(np.zeros((0, B, G * N if k in ("dBm", "dCm") else E)))
    none = Bound(np.zeros((1, B, E)))
    out["dA"] = (stack(rows["dA"]) if T else Bound(np.zeros((1, B, E, N)))).sum((0, 1))
    out["dD"] = (stack(rows["dD"]) if T else none).sum((0, 1))
    out["ddelta_bias"] = (stack(rows["ddelta"]) if T else none).sum((0, 1))
    out["dh0"] = g
    return out
