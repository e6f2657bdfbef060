"""Calls of the state-space block's operators for tests: inputs from a seed, the package's calls on the GPU, the oracle's
values and bounds for the same inputs."""

import numpy as np
import torch

import layer_rnn_forward_amd as R
from oracle import block_oracle as O

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def room(n, fill=0xA5):
    """A workspace whose old contents would show."""
    return torch.full((n,), fill, dtype=torch.uint8, device="cuda")


def numbers(seed, shape, dtype="f32", std=1.0, mean=0.0):
    """A tensor on the host, as the element type holds it."""
    v = np.random.default_rng(seed).normal(size=shape) * std + mean
    return torch.tensor(v).to(DT[dtype])


def host(t):
    return None if t is None else t.double().cpu().numpy()


def gpu(t):
    return None if t is None else t.cuda()


def apart(t, extra, before=0):
    """The same values in a slice of a wider tensor, whose other columns are NaN."""
    w = torch.full(t.shape[:-1] + (t.shape[-1] + extra,), float("nan"), dtype=t.dtype, device=t.device)
    w[..., before:before + t.shape[-1]] = t
    return w[..., before:before + t.shape[-1]]


# -------------------------------------------------------------------- norm
def norm_case(M, D, dtype, seed=0, residual=True, weight=True, bias=True, spread=0.0):
    c = {"x": numbers([seed, 1], (M, D), dtype), "residual": numbers([seed, 2], (M, D), dtype, 3.0) if residual else None,
         "weight": numbers([seed, 3], (D,), "f32", 0.3, 1.0) if weight else None,
         "bias": numbers([seed, 4], (D,), "f32", 0.3) if bias else None,
         "dy": numbers([seed, 5], (M, D), dtype), "dtotal": numbers([seed, 6], (M, D), dtype) if residual else None}
    if spread:
        c["x"] = (c["x"].double() + spread).to(DT[dtype])
    return c


def norm_run(kind, c, eps=1e-5):
    g = {k: gpu(v) for k, v in c.items()}
    x = g["x"]
    M, D = x.shape
    out = {"y": torch.full_like(x, 7.0), "dx": torch.full_like(x, 7.0)}
    total = torch.full_like(x, 7.0) if c["residual"] is not None else None
    stats = torch.full((M, 2), 7.0, device="cuda")
    R.rnn_norm_forward(kind, x, g["residual"], g["weight"], g["bias"], out["y"], total, stats, eps)
    ws = room(R.rnn_norm_workspace_size(M, D) + 64)
    out["dweight"], out["dbias"] = torch.full((D,), 7.0, device="cuda"), torch.full((D,), 7.0, device="cuda")
    R.rnn_norm_backward(kind, x if total is None else total, g["weight"], stats, g["dy"], g["dtotal"], out["dx"],
                        out["dweight"], out["dbias"], ws)
    assert (ws[-64:] == 0xA5).all()
    if total is not None:
        out["total"] = total
    return out


def norm_want(kind, c, eps=1e-5):
    s = host(c["x"])
    out = {}
    if c["residual"] is not None:
        s = (c["x"].double() + c["residual"].double()).float().to(c["x"].dtype)     # fp32's sum, rounded once more
        out["total"], s = s, host(s)
    out["y"] = O.norm_forward(kind, s, host(c["weight"]), host(c["bias"]), eps)[0]
    out["dx"], out["dweight"], out["dbias"] = O.norm_backward(kind, s, host(c["weight"]), eps, host(c["dy"]), host(c["dtotal"]))
    return out


# -------------------------------------------------------------------- conv
def conv_case(T, B, C, K, dtype, lengths=None, seed=0, bias=True, state=True):
    st = (K - 1, B, C)
    return {"x": numbers([seed, 1], (T, B, C), dtype), "w": numbers([seed, 2], (C, K), "f32", K ** -0.5),
            "bias": numbers([seed, 3], (C,), "f32", 0.3) if bias else None,
            "s0": numbers([seed, 4], st, dtype) if state else None, "dy": numbers([seed, 5], (T, B, C), dtype),
            "dsy": numbers([seed, 6], st, dtype) if state else None,
            "lengths": None if lengths is None else torch.tensor(lengths, dtype=torch.int32)}


def conv_run(act, c, wide=0):
    g = {k: gpu(v) for k, v in c.items()}
    T, B, C = c["x"].shape
    K = c["w"].shape[1]
    dt = c["x"].dtype
    st = (K - 1, B, C)
    like = (lambda t: apart(torch.full_like(t, 7.0), wide, wide // 2)) if wide else (lambda t: torch.full_like(t, 7.0))
    if wide:
        g["x"], g["dy"] = apart(g["x"], wide, 1), apart(g["dy"], wide + 2, wide)
    out = {"y": like(gpu(c["x"])), "sy": torch.full(st, 7.0, dtype=dt, device="cuda")}
    R.rnn_conv_forward(act, g["x"], g["w"], g["bias"], g["s0"], g["lengths"], out["y"], out["sy"])
    out |= {"dx": like(gpu(c["x"])), "dw": torch.full((C, K), 7.0, device="cuda"),
            "dbias": torch.full((C,), 7.0, device="cuda"), "ds0": torch.full(st, 7.0, dtype=dt, device="cuda")}
    ws = room(R.rnn_conv_workspace_size(T, B, C, K) + 64)
    R.rnn_conv_backward(act, g["x"], g["w"], g["bias"], g["s0"], g["lengths"], g["dy"], g["dsy"], out["dx"], out["dw"],
                        out["dbias"], out["ds0"], ws)
    assert (ws[-64:] == 0xA5).all()
    return out


def conv_want(act, c):
    lengths = None if c["lengths"] is None else c["lengths"].tolist()
    return O.conv(act, host(c["x"]), host(c["w"]), host(c["bias"]), host(c["s0"]), lengths, host(c["dy"]), host(c["dsy"]))


# --------------------------------------------------------------------- ssm
INPUTS = ("u", "delta", "A", "Bm", "Cm", "D", "z", "delta_bias")


def ssm_case(T, B, E, N, G, dtype, lengths=None, seed=0, mode="softplus", gated=True, extras=True, state=True):
    """Steps between about 0.001 and 1; A between -N and 0, with some rows near 0."""
    c = {"u": numbers([seed, 1], (T, B, E), dtype), "delta": numbers([seed, 2], (T, B, E), dtype, 0.7),
         "A": -(torch.arange(1, N + 1).float() * torch.exp(numbers([seed, 3], (E, N), "f32", 0.5))),
         "Bm": numbers([seed, 4], (T, B, G * N), dtype), "Cm": numbers([seed, 5], (T, B, G * N), dtype),
         "D": numbers([seed, 6], (E,)) if extras else None, "z": numbers([seed, 7], (T, B, E), dtype) if gated else None,
         "delta_bias": numbers([seed, 8], (E,), "f32", 1.5, -3.0) if extras else None,
         "h0": numbers([seed, 9], (B, E, N)) if state else None, "dy": numbers([seed, 10], (T, B, E), dtype),
         "dhy": numbers([seed, 11], (B, E, N)) if state else None,
         "lengths": None if lengths is None else torch.tensor(lengths, dtype=torch.int32)}
    c["A"][::3] *= 0.01
    if mode == "linear":
        c["delta"] = (c["delta"].float().abs() * 0.1).to(DT[dtype])
        if extras:
            c["delta_bias"] = c["delta_bias"].abs() * 0.01
    return c


def ssm_run(mode, c, wide=0, backward=True):
    g = {k: gpu(v) for k, v in c.items()}
    T, B, E = c["u"].shape
    N = c["A"].shape[1]
    G = c["Bm"].shape[2] // N
    like = (lambda t: apart(torch.full_like(t, 7.0), wide, wide // 2)) if wide else (lambda t: torch.full_like(t, 7.0))
    if wide:
        for i, k in enumerate(("u", "delta", "Bm", "Cm", "z", "dy")):
            if g[k] is not None:
                g[k] = apart(g[k], wide + i, i)
    plain = {k: gpu(c[k]) for k in ("u", "Bm")}
    out = {"y": like(plain["u"]), "hy": torch.full((B, E, N), 7.0, device="cuda")}
    save = "full" if backward else "none"
    size = R.rnn_ssm_workspace_size(T, B, E, N, G, save)
    ws = room(size + 64)
    R.rnn_ssm_forward(mode, *(g[k] for k in INPUTS), g["h0"], g["lengths"], out["y"], out["hy"], ws, save)
    if backward:
        out |= {"du": like(plain["u"]), "ddelta": like(plain["u"]), "dBm": like(plain["Bm"]), "dCm": like(plain["Bm"]),
                "dA": torch.full((E, N), 7.0, device="cuda"), "dD": torch.full((E,), 7.0, device="cuda"),
                "ddelta_bias": torch.full((E,), 7.0, device="cuda"), "dh0": torch.full((B, E, N), 7.0, device="cuda")}
        if g["z"] is not None:
            out["dz"] = like(plain["u"])
        R.rnn_ssm_backward(mode, *(g[k] for k in INPUTS), g["h0"], g["lengths"], g["dy"], g["dhy"], out["du"],
                           out["ddelta"], out["dA"], out["dBm"], out["dCm"], out["dD"], out.get("dz"),
                           out["ddelta_bias"], out["dh0"], ws)
    assert (ws[-64:] == 0xA5).all()
    return out


def ssm_want(mode, c, backward=True):
    lengths = None if c["lengths"] is None else c["lengths"].tolist()
    grads = (host(c["dy"]), host(c["dhy"])) if backward else ()
    return O.ssm(mode, *(host(c[k]) for k in INPUTS), host(c["h0"]), lengths, *grads)
