"""The operators of a recurrent language model's block, as workloads: the gated linear recurrence
(scan), the gated feed-forward block and 8-bit activation checkpoints.

Plain forms are elementary torch operations in float32; ``exact`` gives the definition in float64.

Layouts: time-major tensors as in the rest of the package.  The scan's gates ``g`` are [T, B, dirs * 2 * H]
with, for each direction, H columns of the first gate and H of the second; ``y`` is [T, B, dirs * H].  The
feed-forward weights are ``w_in`` [2F, D] (F gate rows, then F up rows) and ``w_out`` [D, F].
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
GROUP = 32      # values of a row that share one power of two in a checkpoint


def _scan(name, kind, T, B, H, dirs, dtype, mode, ragged):
    return {"name": name, "op": "scan", "kind": kind, "T": T, "B": B, "H": H, "dirs": dirs, "dtype": dtype,
            "mode": mode, "ragged": ragged}


def _ffn(name, M, D, F, dtype, act, save):
    return {"name": name, "op": "ffn", "M": M, "D": D, "F": F, "dtype": dtype, "act": act, "save": save}


def _ckpt(name, rows, cols, dtype):
    return {"name": name, "op": "checkpoint", "rows": rows, "cols": cols, "dtype": dtype}


def listed():
    return [
        # one generated token for 16 streams at the Deep Speech 2 width: launch latency
        _scan("scan_token_bf16", "step", 1, 16, 800, 1, "bf16", "gated", False),
        # a packed batch of utterances, both directions, inference in float32
        _scan("scan_packed_infer_f32", "infer", 300, 20, 800, 2, "f32", "gated", True),
        # an ordinary training batch
        _scan("scan_train_bf16", "train", 2048, 8, 1024, 1, "bf16", "gated", False),
        # odd sizes, ragged rows, gates made by the caller
        _scan("scan_train_odd_f32", "train", 1237, 7, 357, 2, "f32", "linear", True),
        # one very long sequence: few rows, the time axis has to be split
        _scan("scan_train_long_bf16", "train", 65536, 1, 1760, 1, "bf16", "gated", False),
        # one generated token: the weights are read once
        _ffn("ffn_token_bf16", 1, 2048, 8192, "bf16", "silu", "none"),
        # inference over a batch of utterances (300 steps of 20 rows)
        _ffn("ffn_infer_bf16", 6000, 800, 3200, "bf16", "gelu", "none"),
        # a large training step
        _ffn("ffn_train_bf16", 8192, 2048, 8192, "bf16", "silu", "full"),
        # a small training step with odd widths in float32
        _ffn("ffn_train_odd_f32", 613, 357, 1021, "f32", "sigmoid", "full"),
        # a training step that keeps its activations in 8 bits
        _ffn("ffn_train_saved8_bf16", 6000, 1760, 7040, "bf16", "silu", "int8"),
        # a small tensor kept and read back: two launches
        _ckpt("checkpoint_small_f32", 20, 800, "f32"),
        # the activations of a long batch
        _ckpt("checkpoint_large_bf16", 65536, 2048, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    what = rng.choice(["step", "infer", "train", "train", "token", "ffn", "ffn", "ffn8", "checkpoint"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if what == "step":
        c = _scan("", "step", 1, _log_int(rng, 1, 256), _log_int(rng, 8, 4096), 1, dtype,
                  rng.choice(["gated", "linear"]), False)
    elif what in ("infer", "train"):
        H, B = _log_int(rng, 8, 4096), _log_int(rng, 1, 64)
        dirs = rng.choice([1, 1, 2])
        most = (1 << 26) // (H * B * dirs)          # below the longest listed sequence's elements
        T = _log_int(rng, 2, max(2, min(65536, most)))
        c = _scan("", what, T, B, H, dirs, dtype, rng.choice(["gated", "linear"]), rng.random() < 0.5)
    elif what == "checkpoint":
        cols = _log_int(rng, 1, 8192)
        c = _ckpt("", _log_int(rng, 1, min(65536, (1 << 26) // cols)), cols, dtype)
    else:
        D, F = _log_int(rng, 64, 4096), _log_int(rng, 64, 8192)
        if rng.random() < 0.6:                       # widths as most models have them
            D, F = -(-D // 8) * 8, -(-F // 8) * 8
        act = rng.choice(["sigmoid", "silu", "gelu"])
        if what == "token":
            c = _ffn("", rng.randint(1, 16), D, F, dtype, act, "none")
        else:
            M = _log_int(rng, 17, max(17, min(16384, (1 << 36) // (D * F))))
            save = "int8" if what == "ffn8" else rng.choice(["none", "full"])
            c = _ffn("", M, D, F, "bf16" if save == "int8" else dtype, act, save)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(mean, std, generator=gen).to(dtype)

    s = dict(case)
    if case["op"] == "scan":
        T, B, H, D = case["T"], case["B"], case["H"], case["dirs"]
        g = torch.empty((T, B, D, 2, H), dtype=dt, device="cuda")
        if case["mode"] == "gated":                  # update gates that lean towards remembering
            g[:, :, :, 0] = normal(T, B, D, H, std=1.5, mean=1.0)
            g[:, :, :, 1] = normal(T, B, D, H)
        else:
            a = torch.sigmoid(normal(T, B, D, H, std=1.5, mean=2.0, dtype=torch.float32))
            g[:, :, :, 0] = a.to(dt)
            g[:, :, :, 1] = ((1 - a) * normal(T, B, D, H, dtype=torch.float32)).to(dt)
        s["g"] = g.view(T, B, D * 2 * H)
        s["h0"] = normal(D, B, H, std=0.5, dtype=torch.float32)
        s["lengths"] = None
        if case["ragged"]:                           # whole rows, short rows and empty ones
            n = torch.randint(0, T + 1, (B,), device="cuda", generator=gen)
            n[0] = T
            s["lengths"] = n.to(torch.int32)
        if case["kind"] == "train":
            s["dy"] = normal(T, B, D * H)
            s["dhy"] = normal(D, B, H, dtype=torch.float32)
    elif case["op"] == "ffn":
        M, D, F = case["M"], case["D"], case["F"]
        s["x"] = normal(M, D)
        s["w_in"] = normal(2 * F, D, std=D ** -0.5)
        s["w_out"] = normal(D, F, std=F ** -0.5)
        if case["save"] != "none":
            s["dy"] = normal(M, D)
    else:                                            # rows of different sizes, a few values far out
        x = normal(case["rows"], case["cols"], dtype=torch.float32)
        x *= torch.exp2(normal(case["rows"], 1, std=2.0, dtype=torch.float32))
        s["x"] = (x * (1 + 20 * (normal(case["rows"], case["cols"], dtype=torch.float32) > 3.5))).to(dt)
    return s


# -------------------------------------------------------------- plain forms
def _plain_recurrence(a, b, h0):
    """h[t] = a[t] h[t-1] + b[t] over the first axis by doubling: after the pass with distance k every
    position holds the composition of its last 2k steps."""
    h = b.clone()
    h[0] += a[0] * h0
    a, k, T = a.clone(), 1, a.shape[0]
    while k < T:
        h[k:] = torch.addcmul(h[k:], a[k:], h[:-k])
        a[k:] = a[k:] * a[:-k]
        k *= 2
    return h


def _in_order(v):
    """[T, B, dirs, H] with the second direction's steps in the order it walks them."""
    return v if v.shape[2] == 1 else torch.cat([v[:, :, :1], v[:, :, 1:].flip(0)], 2)


def _plain_scan(s):
    T, B, H, D = s["T"], s["B"], s["H"], s["dirs"]
    g = s["g"].view(T, B, D, 2, H).float()
    p, q = _in_order(g[:, :, :, 0]), _in_order(g[:, :, :, 1])
    valid = None
    if s["lengths"] is not None:
        t = torch.arange(T, device=g.device)[:, None]
        valid = _in_order((t < s["lengths"][None]).view(T, B, 1, 1).expand(T, B, D, 1))
    if s["mode"] == "gated":
        z, n = torch.sigmoid(p), torch.tanh(q)
        a, b = z, torch.sigmoid(-p) * n
    else:
        a, b = p, q
    if valid is not None:
        a, b = torch.where(valid, a, 1.0), torch.where(valid, b, 0.0)
    h0 = s["h0"].transpose(0, 1)
    h = _plain_recurrence(a, b, h0)
    y = h if valid is None else torch.where(valid, h, 0.0)
    dt = s["g"].dtype
    out = {"y": _in_order(y).reshape(T, B, D * H).to(dt), "hy": h[-1].transpose(0, 1).contiguous()}
    if s["kind"] != "train":
        return out
    dy = _in_order(s["dy"].view(T, B, D, H).float())
    if valid is not None:
        dy = torch.where(valid, dy, 0.0)
    nxt = torch.cat([a[1:], torch.ones_like(a[:1])])
    dh = _plain_recurrence(nxt.flip(0), dy.flip(0), s["dhy"].transpose(0, 1)).flip(0)
    before = torch.cat([h0[None], h[:-1]])
    if s["mode"] == "gated":
        dp, dq = dh * (before - n) * z * torch.sigmoid(-p), dh * torch.sigmoid(-p) * (1 - n * n)
    else:
        dp, dq = dh * before, dh
    if valid is not None:
        dp, dq = torch.where(valid, dp, 0.0), torch.where(valid, dq, 0.0)
    out["dg"] = torch.stack([_in_order(dp), _in_order(dq)], 3).reshape(T, B, D * 2 * H).to(dt)
    out["dh0"] = (a[0] * dh[0]).transpose(0, 1).contiguous()
    return out


def _plain_act(name, g):
    """act(g) and its derivative."""
    if name == "gelu":                               # the tanh form
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    sg = torch.sigmoid(g)
    return (sg, sg * (1 - sg)) if name == "sigmoid" else (g * sg, sg * (1 + g * (1 - sg)))


def _plain_round8(x):
    """x as a checkpoint holds it: 8-bit whole numbers times a power of two for each group of a row."""
    R, C = x.shape
    v = torch.nn.functional.pad(x, (0, -C % GROUP)).view(R, -1, GROUP)
    e = (torch.frexp(v.abs().amax(2, keepdim=True))[1] - 7).clamp(min=-126)
    q = torch.round(torch.ldexp(v, -e)).clamp(-127, 127)
    return torch.ldexp(q, e).view(R, -1)[:, :C]


def _plain_ffn(s):
    x, w_in, w_out, F, dt = s["x"].float(), s["w_in"].float(), s["w_out"].float(), s["F"], s["x"].dtype
    gu = x @ w_in.T
    g, u = gu[:, :F], gu[:, F:]
    h = _plain_act(s["act"], g)[0] * u
    out = {"y": (h @ w_out.T).to(dt)}
    if s["save"] == "none":
        return out
    if s["save"] == "int8":
        x, g, u = _plain_round8(x), _plain_round8(g), _plain_round8(u)
    a, da = _plain_act(s["act"], g)
    dy = s["dy"].float()
    dh = dy @ w_out
    dgu = torch.cat([dh * u * da, dh * a], 1)
    out["dx"] = (dgu @ w_in).to(dt)
    out["dw_in"] = (dgu.T @ x).to(dt)
    out["dw_out"] = (dy.T @ (a * u)).to(dt)
    return out


# ------------------------------------------------------- the package's calls
def _own_scan(s):
    import layer_rnn_forward_amd as R
    T, B, H, D, dt = s["T"], s["B"], s["H"], s["dirs"], s["g"].dtype
    y = torch.empty((T, B, D * H), dtype=dt, device="cuda")
    if s["kind"] == "step":
        hy = torch.empty_like(s["h0"])
        R.rnn_scan_step(s["mode"], s["g"][0], s["h0"][0], y[0], hy[0])
        return {"y": y, "hy": hy}
    if "ws" not in s:                                # the workspace a program keeps between its passes
        s["ws"] = torch.empty(R.rnn_scan_workspace_size(T, B, H, D), dtype=torch.uint8, device="cuda")
    hy = torch.empty_like(s["h0"])
    R.rnn_scan_forward(s["mode"], s["g"], s["h0"], s["lengths"], y, hy, s["ws"])
    out = {"y": y, "hy": hy}
    if s["kind"] == "train":
        out["dg"], out["dh0"] = torch.empty_like(s["g"]), torch.empty_like(s["h0"])
        R.rnn_scan_backward(s["mode"], s["g"], s["h0"], s["lengths"], s["dy"], s["dhy"], out["dg"], out["dh0"],
                            s["ws"])
    return out


def _own_ffn(s):
    import layer_rnn_forward_amd as R
    M, D, F, dt = s["M"], s["D"], s["F"], s["dtype"]
    if "ws" not in s:                                # kept between passes: scratch, and what backward reads
        s["ws"] = torch.empty(R.rnn_ffn_workspace_size(M, D, F, dt, s["save"]), dtype=torch.uint8, device="cuda")
        s["reserve"] = torch.empty(R.rnn_ffn_reserve_size(M, D, F, dt, s["save"]), dtype=torch.uint8, device="cuda")
    out = {"y": torch.empty_like(s["x"])}
    R.rnn_ffn_forward(s["act"], s["x"], s["w_in"], s["w_out"], out["y"], s["ws"], s["save"], s["reserve"])
    if s["save"] == "none":
        return out
    out["dx"] = torch.empty_like(s["x"])
    out["dw_in"], out["dw_out"] = torch.empty_like(s["w_in"]), torch.empty_like(s["w_out"])
    R.rnn_ffn_backward(s["act"], None if s["save"] == "int8" else s["x"], s["w_in"], s["w_out"], s["dy"],
                       out["dx"], out["dw_in"], out["dw_out"], s["ws"], s["save"], s["reserve"])
    return out


def _own_checkpoint(s):
    import layer_rnn_forward_amd as R
    kept = torch.empty(R.rnn_checkpoint_size(s["rows"], s["cols"]), dtype=torch.uint8, device="cuda")
    R.rnn_checkpoint_store(s["x"], kept)
    back = torch.empty_like(s["x"])
    R.rnn_checkpoint_load(kept, back)
    return {"x": back}


def run(state):
    if own:
        return {"scan": _own_scan, "ffn": _own_ffn, "checkpoint": _own_checkpoint}[state["op"]](state)
    if state["op"] == "scan":
        return _plain_scan(state)
    if state["op"] == "ffn":
        return _plain_ffn(state)
    return {"x": _plain_round8(state["x"].float()).to(state["x"].dtype)}


# ---------------------------------------------------------------- the work
def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "scan":
        n = case["T"] * case["B"] * case["H"] * case["dirs"]
        st = case["B"] * case["H"] * case["dirs"] * 4
        if case["kind"] == "train":                  # in: g, dy, h0, dhy; out: y, dg, hy, dh0
            return {"bytes": 6 * n * es + 4 * st, "flops": 30 * n}
        return {"bytes": 3 * n * es + 2 * st, "flops": 10 * n}
    if case["op"] == "ffn":
        M, D, F = case["M"], case["D"], case["F"]
        b = es * (2 * M * D + 3 * D * F)
        if case["save"] != "none":
            b += es * (2 * M * D + 3 * D * F)
        return {"bytes": b, "flops": (6 if case["save"] == "none" else 18) * M * D * F}
    n = case["rows"] * case["cols"]
    return {"bytes": 2 * n * es + n + case["rows"] * -(-case["cols"] // GROUP), "flops": 4 * n}


# ---------------------------------------------- the definitions in 64 bits
def _exact_scan(s):
    T, B, H, D = s["T"], s["B"], s["H"], s["dirs"]
    g = s["g"].double().view(T, B, D, 2, H)
    first, second = g[:, :, :, 0], g[:, :, :, 1]
    gated = s["mode"] == "gated"
    if gated:
        keep, cand = 1 / (1 + torch.exp(-first)), torch.tanh(second)
        add = cand / (1 + torch.exp(first))
    else:
        keep, add = first.clone(), second.clone()
    n = torch.full((B,), T, device=g.device) if s["lengths"] is None else s["lengths"].long().clamp(0, T)
    live = (torch.arange(T, device=g.device)[:, None] < n[None]).double()[:, :, None]
    train = s["kind"] == "train"
    y = torch.zeros(T, B, D, H, dtype=torch.float64, device=g.device)
    dg = torch.zeros(T, B, D, 2, H, dtype=torch.float64, device=g.device) if train else None
    hy, dh0 = torch.empty(D, B, H, dtype=torch.float64, device=g.device), None
    if train:
        dh0 = torch.empty_like(hy)
    for d in range(D):
        k, c = keep[:, :, d] * live + (1 - live), add[:, :, d] * live
        steps = range(T) if d == 0 else range(T - 1, -1, -1)
        h = s["h0"][d].double()
        before = torch.empty(T, B, H, dtype=torch.float64, device=g.device)
        for t in steps:
            before[t] = h
            h = torch.addcmul(c[t], k[t], h)
            y[t, :, d] = h
        hy[d] = h
        if train:
            up = s["dy"].double().view(T, B, D, H)[:, :, d] * live
            dh, dhs = s["dhy"][d].double(), torch.empty(T, B, H, dtype=torch.float64, device=g.device)
            for t in reversed(steps):
                dh = up[t] + dh
                dhs[t] = dh
                dh = dh * k[t]
            dh0[d] = dh
            dhs *= live
            if gated:
                kk, cc = keep[:, :, d], cand[:, :, d]
                dg[:, :, d, 0] = dhs * (before - cc) * kk * (1 - kk)
                dg[:, :, d, 1] = dhs * (1 - kk) * (1 - cc ** 2)
            else:
                dg[:, :, d, 0], dg[:, :, d, 1] = dhs * before, dhs
    y *= live[:, :, :, None]
    out = {"y": y.view(T, B, D * H), "hy": hy}
    if train:
        out["dg"], out["dh0"] = dg.view(T, B, D * 2 * H), dh0
    return out


def _exact_round8(x):
    out = torch.empty_like(x)
    for c in range(0, x.shape[1], GROUP):
        v = x[:, c:c + GROUP]
        top = v.abs().max(1, keepdim=True).values
        e = torch.where(top > 0, torch.floor(torch.log2(top.clamp(min=2.0 ** -1000))), -126.0)
        e = e + (torch.exp2(e + 1) <= top).double() - (torch.exp2(e) > top).double() * (top > 0)
        unit = torch.exp2(torch.clamp(e - 6, min=-126.0))
        out[:, c:c + GROUP] = torch.clamp(torch.round(v / unit), -127, 127) * unit
    return out


def _exact_act(name, g):
    g = g.detach().requires_grad_(True)
    if name == "gelu":
        a = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    else:
        a = (g if name == "silu" else 1) / (1 + torch.exp(-g))
    return a.detach(), torch.autograd.grad(a.sum(), g)[0]


def _exact_ffn(s):
    F, x = s["F"], s["x"].double()
    wg, wu, wo = s["w_in"][:F].double(), s["w_in"][F:].double(), s["w_out"].double()
    g, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
    y = torch.mm(_exact_act(s["act"], g)[0] * u, wo.t())
    if s["save"] == "none":
        return {"y": y}
    if s["save"] == "int8":
        x, g, u = _exact_round8(x), _exact_round8(g), _exact_round8(u)
    a, slope = _exact_act(s["act"], g)
    dy = s["dy"].double()
    dh = torch.mm(dy, wo)
    dg, du = dh * u * slope, dh * a
    return {"y": y, "dx": torch.mm(dg, wg) + torch.mm(du, wu),
            "dw_in": torch.cat([torch.mm(dg.t(), x), torch.mm(du.t(), x)]), "dw_out": torch.mm(dy.t(), a * u)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "scan":
        return _exact_scan(s)
    if case["op"] == "ffn":
        return _exact_ffn(s)
    return {"x": _exact_round8(s["x"].double())}
