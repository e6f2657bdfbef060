"""The operators of a selective state-space language model's block, as workloads: normalisation of rows with the
residual addition before it, the short causal convolution, and the selective state-space scan.

Plain forms are elementary torch operations in float32; ``exact`` gives the definition in float64.

Layouts: time-major as in the rest of the package.  The normalisation takes rows [M, D].  The convolution's input is
[T, B, C], its weights [C, K] with the newest input's last, its states the K - 1 inputs before the first and after
the last step [K - 1, B, C].  The state-space scan takes ``u``, ``delta``, ``z`` [T, B, E], ``Bm`` and ``Cm``
[T, B, G * N] (G groups of E / G neighbouring channels), ``A`` [E, N], ``D`` and ``delta_bias`` [E], and states
[B, E, N].  Inputs that a block's projections make side by side are slices of one tensor.  Parameters, states and
the parameters' gradients are float32.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


def _norm(name, kind, M, D, dtype, mode, residual):
    return {"name": name, "op": "norm", "kind": kind, "M": M, "D": D, "dtype": dtype, "mode": mode,
            "residual": residual}


def _conv(name, kind, T, B, C, K, dtype, act, ragged):
    return {"name": name, "op": "conv", "kind": kind, "T": T, "B": B, "C": C, "K": K, "dtype": dtype, "act": act,
            "ragged": ragged}


def _ssm(name, kind, T, B, E, N, groups, dtype, ragged):
    return {"name": name, "op": "ssm", "kind": kind, "T": T, "B": B, "E": E, "N": N, "groups": groups,
            "dtype": dtype, "ragged": ragged}


def listed():
    return [
        # one generated token for 16 streams: the residual stream is added to and normalised, launch latency
        _norm("norm_token_bf16", "infer", 16, 2048, "bf16", "rms", True),
        # a training batch of 8 rows of 2048 steps
        _norm("norm_train_bf16", "train", 16384, 2048, "bf16", "rms", True),
        # odd sizes, mean and bias, no residual
        _norm("norm_train_odd_f32", "train", 4291, 1357, "f32", "layer", False),
        # one generated token for 16 streams
        _conv("conv_token_bf16", "step", 1, 16, 1600, 4, "bf16", "silu", False),
        # a training batch
        _conv("conv_train_bf16", "train", 2048, 8, 2048, 4, "bf16", "silu", False),
        # odd sizes, ragged rows, no activation
        _conv("conv_train_odd_f32", "train", 1237, 7, 357, 3, "f32", "none", True),
        # one generated token for 16 streams
        _ssm("ssm_token_bf16", "step", 1, 16, 1600, 16, 1, "bf16", False),
        # the prompt of one stream
        _ssm("ssm_prompt_bf16", "infer", 8192, 1, 3520, 16, 1, "bf16", False),
        # a packed batch of prompts in float32, ragged
        _ssm("ssm_prompts_f32", "infer", 300, 20, 1600, 16, 1, "f32", True),
        # a training batch
        _ssm("ssm_train_bf16", "train", 2048, 8, 2048, 16, 1, "bf16", False),
        # odd sizes, ragged rows, several groups
        _ssm("ssm_train_odd_f32", "train", 613, 5, 357, 13, 3, "f32", True),
        # training on one long sequence: few rows, the time axis has to be split
        _ssm("ssm_train_long_bf16", "train", 16384, 1, 1760, 16, 1, "bf16", False),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "conv", "ssm", "ssm"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        D = _log_int(rng, 32, 8192)
        if rng.random() < 0.6:                       # widths as most models have them
            D = -(-D // 8) * 8
        M = _log_int(rng, 1, min(16384, (1 << 25) // D))
        c = _norm("", rng.choice(["infer", "train"]), M, D, dtype, rng.choice(["rms", "layer"]), rng.random() < 0.6)
    elif op == "conv":
        kind, C, B, K = rng.choice(["step", "infer", "train"]), _log_int(rng, 16, 4096), _log_int(rng, 1, 32), rng.randint(2, 6)
        if rng.random() < 0.6:
            C = -(-C // 8) * 8
        T = 1 if kind == "step" else _log_int(rng, 1, max(1, min(32768, (1 << 25) // (B * C))))
        c = _conv("", kind, T, B, C, K, dtype, rng.choice(["silu", "silu", "none"]), kind != "step" and rng.random() < 0.5)
    else:
        kind, B, N = rng.choice(["step", "infer", "train", "train"]), _log_int(rng, 1, 32), rng.choice([4, 8, 13, 16, 16, 16, 24, 32])
        G = rng.choice([1, 1, 1, 2, 4])
        E = G * _log_int(rng, 16, 4096 // G)
        if rng.random() < 0.6:
            E = -(-E // (8 * G)) * 8 * G
        T = 1 if kind == "step" else _log_int(rng, 1, max(1, min(16384, (1 << 28) // (B * E * N))))
        c = _ssm("", kind, T, B, E, N, G, dtype, kind != "step" and rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(mean, std, generator=gen).to(dtype)

    def lengths(T, B):                               # whole rows, short rows and empty ones
        if not case["ragged"]:
            return None
        n = torch.randint(0, T + 1, (B,), device="cuda", generator=gen)
        n[0] = T
        return n.to(torch.int32)

    s = dict(case)
    train = case["kind"] == "train"
    if case["op"] == "norm":
        M, D = case["M"], case["D"]
        s["x"] = normal(M, D, dtype=dt)
        s["residual"] = normal(M, D, std=3.0, dtype=dt) if case["residual"] else None
        s["weight"] = normal(D, std=0.1, mean=1.0)
        s["bias"] = normal(D, std=0.1) if case["mode"] == "layer" else None
        if train:
            s["dy"] = normal(M, D, dtype=dt)
            s["dtotal"] = normal(M, D, dtype=dt) if case["residual"] else None
    elif case["op"] == "conv":
        T, B, C, K = case["T"], case["B"], case["C"], case["K"]
        s["xz"] = normal(T, B, 2 * C, dtype=dt)      # the block's input projection: the convolution's half and the gate's
        s["x"] = s["xz"][:, :, :C]
        s["w"] = normal(C, K, std=K ** -0.5)
        s["bias"] = normal(C, std=0.1)
        s["s0"] = normal(K - 1, B, C, dtype=dt)
        s["lengths"] = lengths(T, B)
        if train:
            s["dy"], s["dsy"] = normal(T, B, C, dtype=dt), normal(K - 1, B, C, dtype=dt)
    else:
        T, B, E, N, G = case["T"], case["B"], case["E"], case["N"], case["groups"]
        s["u"] = torch.nn.functional.silu(normal(T, B, E)).to(dt)
        s["xz"] = normal(T, B, 2 * E, dtype=dt)
        s["z"] = s["xz"][:, :, E:]
        s["delta"] = normal(T, B, E, std=0.5, dtype=dt)
        s["bc"] = normal(T, B, 2 * G * N, dtype=dt)
        s["Bm"], s["Cm"] = s["bc"][:, :, :G * N], s["bc"][:, :, G * N:]
        s["A"] = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * torch.exp(normal(E, N, std=0.1))
        s["D"] = normal(E, std=0.1, mean=1.0)
        step = torch.exp(torch.empty(E, device="cuda").uniform_(math.log(1e-3), math.log(1e-1), generator=gen))
        s["delta_bias"] = step + torch.log(-torch.expm1(-step))      # softplus of it is a step between 0.001 and 0.1
        s["h0"] = normal(B, E, N, std=0.5)
        s["lengths"] = lengths(T, B)
        if train:
            s["dy"], s["dhy"] = normal(T, B, E, dtype=dt), normal(B, E, N)
    return s


# -------------------------------------------------------------- plain forms
def _plain_norm(s):
    dt, x = s["x"].dtype, s["x"].float()
    out = {}
    if s["residual"] is not None:                    # the residual stream is kept in the element type
        x = (x + s["residual"].float()).to(dt)
        out["total"] = x
        x = x.float()
    c = x - x.mean(1, keepdim=True) if s["mode"] == "layer" else x
    rstd = 1 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
    n = c * rstd
    y = n * s["weight"]
    if s["bias"] is not None:
        y = y + s["bias"]
    out["y"] = y.to(dt)
    if s["kind"] != "train":
        return out
    dy = s["dy"].float()
    g = dy * s["weight"]
    dx = g - n * (g * n).mean(1, keepdim=True)
    if s["mode"] == "layer":
        dx = dx - g.mean(1, keepdim=True)
    dx = dx * rstd
    if s["dtotal"] is not None:
        dx = dx + s["dtotal"].float()
    out["dx"], out["dweight"] = dx.to(dt), (dy * n).sum(0)
    if s["bias"] is not None:
        out["dbias"] = dy.sum(0)
    return out


def _valid(s):
    if s["lengths"] is None:
        return None
    return (torch.arange(s["T"], device="cuda")[:, None] < s["lengths"][None])[:, :, None]


def _plain_conv(s):
    dt, T, B, C, K = s["x"].dtype, s["T"], s["B"], s["C"], s["K"]
    valid = _valid(s)
    xs = torch.cat([s["s0"], s["x"]]).float()        # xs[t + K - 1] is step t
    windows = xs.unfold(0, K, 1)                     # [T, B, C, K]
    v = (windows * s["w"]).sum(3) + s["bias"]
    sg = torch.sigmoid(v)
    y = v * sg if s["act"] == "silu" else v
    if valid is not None:
        y = torch.where(valid, y, 0.0)
        last = (s["lengths"][None].long() + torch.arange(K - 1, device="cuda")[:, None])[:, :, None].expand(K - 1, B, C)
        sy = torch.gather(xs, 0, last)
    else:
        sy = xs[T:]
    out = {"y": y.to(dt), "sy": sy.to(dt)}
    if s["kind"] != "train":
        return out
    dv = s["dy"].float()
    if s["act"] == "silu":
        dv = dv * sg * (1 + v * (1 - sg))
    if valid is not None:
        dv = torch.where(valid, dv, 0.0)
    none = torch.zeros(K - 1, B, C, device="cuda")
    dxs = (torch.cat([none, dv, none]).unfold(0, K, 1) * s["w"].flip(1)).sum(3)
    dsy = s["dsy"].float()
    if valid is not None:
        dxs = dxs.scatter_add(0, last, dsy)
    else:
        dxs[T:] += dsy
    out["dx"], out["ds0"] = dxs[K - 1:].to(dt), dxs[:K - 1].to(dt)
    out["dw"], out["dbias"] = (windows * dv[..., None]).sum((0, 1)), dv.sum((0, 1))
    return out


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


def _plain_ssm(s):
    dt, T, B, E, N, G = s["u"].dtype, s["T"], s["B"], s["E"], s["N"], s["groups"]
    valid = _valid(s)
    u, z, A = s["u"].float(), s["z"].float(), s["A"]
    pre = s["delta"].float() + s["delta_bias"]
    step = torch.clamp(pre, min=0) + torch.log1p(torch.exp(-torch.abs(pre)))
    if valid is not None:
        step = torch.where(valid, step, 0.0)

    def states(v):                                   # [T, B, G N] -> [T, B, E, N]
        return v.float().view(T, B, G, 1, N).expand(T, B, G, E // G, N).reshape(T, B, E, N)

    a = torch.exp(step[..., None] * A)
    h = _plain_recurrence(a, (step * u)[..., None] * states(s["Bm"]), s["h0"])
    o = (h * states(s["Cm"])).sum(3) + s["D"] * u
    gate = z * torch.sigmoid(z)
    y = o * gate
    if valid is not None:
        y = torch.where(valid, y, 0.0)
    out = {"y": y.to(dt), "hy": h[-1].clone()}
    if s["kind"] != "train":
        return out
    dy = s["dy"].float()
    if valid is not None:
        dy = torch.where(valid, dy, 0.0)
    sz = torch.sigmoid(z)
    out["dz"] = (dy * o * sz * (1 + z * (1 - sz))).to(dt)
    do = dy * gate

    def grouped(v):                                  # [T, B, E, N] -> [T, B, G N]
        return v.view(T, B, G, E // G, N).sum(3).reshape(T, B, G * N)

    out["dCm"] = grouped(do[..., None] * h).to(dt)
    before = torch.cat([s["h0"][None], h[:-1]])
    del h
    later = torch.cat([a[1:], torch.ones_like(a[:1])])
    dh = _plain_recurrence(later.flip(0), (do[..., None] * states(s["Cm"])).flip(0), s["dhy"]).flip(0)
    out["dh0"] = a[0] * dh[0]
    out["dBm"] = grouped(dh * (step * u)[..., None]).to(dt)
    through = dh * a * before                        # of step A
    del a, before, later
    out["dA"] = (through * step[..., None]).sum((0, 1))
    db = (dh * states(s["Bm"])).sum(3)
    dstep = (through * A).sum(3) + db * u
    dpre = dstep * torch.sigmoid(pre)
    if valid is not None:
        dpre = torch.where(valid, dpre, 0.0)
    out["du"] = (db * step + do * s["D"]).to(dt)
    out["ddelta"], out["ddelta_bias"] = dpre.to(dt), dpre.sum((0, 1))
    out["dD"] = (do * u).sum((0, 1))
    return out


# ------------------------------------------------------- the package's calls
def _own_norm(s):
    import layer_rnn_forward_amd as R
    x, train = s["x"], s["kind"] == "train"
    out = {"y": torch.empty_like(x)}
    if s["residual"] is not None:
        out["total"] = torch.empty_like(x)
    stats = torch.empty((s["M"], 2), device="cuda") if train else None
    R.rnn_norm_forward(s["mode"], x, s["residual"], s["weight"], s["bias"], out["y"], out.get("total"), stats, EPS)
    if not train:
        return out
    if "ws" not in s:                                # the scratch a program keeps between its passes
        s["ws"] = torch.empty(R.rnn_norm_workspace_size(s["M"], s["D"]), dtype=torch.uint8, device="cuda")
    out["dx"], out["dweight"] = torch.empty_like(x), torch.empty_like(s["weight"])
    if s["bias"] is not None:
        out["dbias"] = torch.empty_like(s["bias"])
    R.rnn_norm_backward(s["mode"], out.get("total", x), s["weight"], stats, s["dy"], s["dtotal"], out["dx"],
                        out["dweight"], out.get("dbias"), s["ws"])
    return out


def _own_conv(s):
    import layer_rnn_forward_amd as R
    T, B, C, K, dt = s["T"], s["B"], s["C"], s["K"], s["x"].dtype
    out = {"y": torch.empty((T, B, C), dtype=dt, device="cuda"), "sy": torch.empty_like(s["s0"])}
    if s["kind"] == "step":
        R.rnn_conv_step(s["act"], s["x"][0], s["w"], s["bias"], s["s0"], out["y"][0], out["sy"])
        return out
    R.rnn_conv_forward(s["act"], s["x"], s["w"], s["bias"], s["s0"], s["lengths"], out["y"], out["sy"])
    if s["kind"] != "train":
        return out
    if "ws" not in s:
        s["ws"] = torch.empty(R.rnn_conv_workspace_size(T, B, C, K), dtype=torch.uint8, device="cuda")
    out["dx"], out["ds0"] = torch.empty_like(out["y"]), torch.empty_like(s["s0"])
    out["dw"], out["dbias"] = torch.empty_like(s["w"]), torch.empty_like(s["bias"])
    R.rnn_conv_backward(s["act"], s["x"], s["w"], s["bias"], s["s0"], s["lengths"], s["dy"], s["dsy"], out["dx"],
                        out["dw"], out["dbias"], out["ds0"], s["ws"])
    return out


def _own_ssm(s):
    import layer_rnn_forward_amd as R
    T, B, E, N, G = s["T"], s["B"], s["E"], s["N"], s["groups"]
    out = {"y": torch.empty_like(s["u"]), "hy": torch.empty_like(s["h0"])}
    if s["kind"] == "step":
        R.rnn_ssm_step("softplus", s["u"][0], s["delta"][0], s["A"], s["Bm"][0], s["Cm"][0], s["D"], s["z"][0],
                       s["delta_bias"], s["h0"], out["y"][0], out["hy"])
        return out
    save = "full" if s["kind"] == "train" else "none"
    if "ws" not in s:
        s["ws"] = torch.empty(R.rnn_ssm_workspace_size(T, B, E, N, G, save), dtype=torch.uint8, device="cuda")
    R.rnn_ssm_forward("softplus", s["u"], s["delta"], s["A"], s["Bm"], s["Cm"], s["D"], s["z"], s["delta_bias"],
                      s["h0"], s["lengths"], out["y"], out["hy"], s["ws"], save)
    if s["kind"] != "train":
        return out
    for name in ("du", "ddelta"):
        out[name] = torch.empty_like(s["u"])
    out["dz"] = torch.empty_like(out["y"])
    dbc = torch.empty_like(s["bc"])                  # side by side again, as the projection's gradient wants them
    out["dBm"], out["dCm"] = dbc[:, :, :G * N], dbc[:, :, G * N:]
    for name in ("A", "D", "delta_bias", "h0"):
        out["d" + name] = torch.empty_like(s[name])
    R.rnn_ssm_backward("softplus", s["u"], s["delta"], s["A"], s["Bm"], s["Cm"], s["D"], s["z"], s["delta_bias"],
                       s["h0"], s["lengths"], s["dy"], s["dhy"], out["du"], out["ddelta"], out["dA"], out["dBm"],
                       out["dCm"], out["dD"], out["dz"], out["ddelta_bias"], out["dh0"], s["ws"])
    return out


def run(state):
    if own:
        return {"norm": _own_norm, "conv": _own_conv, "ssm": _own_ssm}[state["op"]](state)
    return {"norm": _plain_norm, "conv": _plain_conv, "ssm": _plain_ssm}[state["op"]](state)


# ---------------------------------------------------------------- the work
def work(case):
    es, train = 2 if case["dtype"] == "bf16" else 4, case["kind"] == "train"
    if case["op"] == "norm":
        M, D = case["M"], case["D"]
        n, vectors = 4 if case["residual"] else 2, 1 if case["mode"] == "rms" else 2
        if train:                                    # and dy, dtotal, dx, the parameters' gradients
            n, vectors = n + (3 if case["residual"] else 2), 2 * vectors
        return {"bytes": n * M * D * es + 4 * vectors * D, "flops": (22 if train else 8) * M * D}
    if case["op"] == "conv":
        T, B, C, K = case["T"], case["B"], case["C"], case["K"]
        n, states, params = 2 * T, 2 * (K - 1), (K + 1) * C * 4
        if train:                                    # and dy, dx, dsy, ds0, dw, dbias
            n, states, params = 2 * n, 2 * states, 2 * params
        return {"bytes": (n + states) * B * C * es + params, "flops": (6 if train else 2) * T * B * C * K}
    T, B, E, N, G = case["T"], case["B"], case["E"], case["N"], case["groups"]
    n, bc, states, params = 4 * T * B * E, 2 * T * B * G * N, 2 * B * E * N * 4, (E * N + 2 * E) * 4
    if train:                                        # and dy, du, ddelta, dz, dBm, dCm, dhy, dh0, dA, dD, ddelta_bias
        n, bc, states, params = 2 * n, 2 * bc, 2 * states, 2 * params
    return {"bytes": (n + bc) * es + states + params, "flops": (28 if train else 7) * T * B * E * N}


# ---------------------------------------------- the definitions in 64 bits
def _exact_norm(s):
    x, dt = s["x"].double(), s["x"].dtype
    out = {}
    if s["residual"] is not None:                    # what is normalised is the sum as the element type holds it
        x = (x + s["residual"].double()).to(dt).double()
        out["total"] = x
    x = x.requires_grad_(True)
    w = s["weight"].double().requires_grad_(True)
    b = s["bias"].double().requires_grad_(True) if s["bias"] is not None else None
    mean = x.sum(1, keepdim=True) / x.shape[1] if s["mode"] == "layer" else 0.0
    var = torch.square(x - mean).sum(1, keepdim=True) / x.shape[1]
    y = (x - mean) * torch.pow(var + EPS, -0.5) * w + (b if b is not None else 0.0)
    out["y"] = y.detach()
    if s["kind"] == "train":
        grads = torch.autograd.grad(y, [x, w] + ([b] if b is not None else []), s["dy"].double())
        out["dx"] = grads[0] + (s["dtotal"].double() if s["dtotal"] is not None else 0.0)
        out["dweight"] = grads[1]
        if b is not None:
            out["dbias"] = grads[2]
    if "total" in out:
        out["total"] = out["total"].detach()
    return out


def _exact_conv(s):
    T, B, K = s["T"], s["B"], s["K"]
    x, s0 = s["x"].double().requires_grad_(True), s["s0"].double().requires_grad_(True)
    w, bias = s["w"].double().requires_grad_(True), s["bias"].double().requires_grad_(True)
    n = [T] * B if s["lengths"] is None else s["lengths"].tolist()
    xs = torch.cat([s0, x])
    v = bias.expand_as(x)
    for k in range(K):
        v = v + w[:, k] * xs[k:k + T]
    y = v / (1 + torch.exp(-v)) if s["act"] == "silu" else v
    live = torch.tensor([[t < m for m in n] for t in range(T)], device="cuda", dtype=torch.float64)[:, :, None]
    y = y * live
    sy = torch.stack([xs[m:m + K - 1, b] for b, m in enumerate(n)], 1)
    out = {"y": y.detach(), "sy": sy.detach()}
    if s["kind"] == "train":
        grads = torch.autograd.grad((y, sy), (x, s0, w, bias), (s["dy"].double(), s["dsy"].double()))
        out.update(zip(("dx", "ds0", "dw", "dbias"), grads))
    return out


def _exact_ssm(s):
    T, B, E, N, G = s["T"], s["B"], s["E"], s["N"], s["groups"]
    train = s["kind"] == "train"
    n = torch.full((B,), T, device="cuda") if s["lengths"] is None else s["lengths"].long()
    A, D = s["A"].double(), s["D"].double()

    def at(v, t):                                    # a step's [B, G N] as [B, G, 1, N]
        return v[t].double().view(B, G, 1, N)

    h = s["h0"].double()
    y, before = torch.zeros(T, B, E, dtype=torch.float64, device="cuda"), []
    steps, os = [], []
    for t in range(T):
        live = (t < n).double()[:, None]
        pre = s["delta"][t].double() + s["delta_bias"].double()
        d = torch.where(pre > 30, pre, torch.log(1 + torch.exp(pre.clamp(max=30)))) * live
        if train:
            before.append(h)
        u = s["u"][t].double()
        h = h * torch.exp(d[..., None] * A) + ((d * u).view(B, G, -1, 1) * at(s["Bm"], t)).view(B, E, N)
        o = (h.view(B, G, -1, N) * at(s["Cm"], t)).sum(3).view(B, E) + D * u
        z = s["z"][t].double()
        y[t] = o * z / (1 + torch.exp(-z)) * live
        if train:
            steps.append(d)
            os.append(o)
    out = {"y": y, "hy": h}
    if not train:
        return out
    du, ddelta, dz = torch.zeros_like(y), torch.zeros_like(y), torch.zeros_like(y)
    dBm, dCm = (torch.zeros(T, B, G * N, dtype=torch.float64, device="cuda") for _ in range(2))
    dA, dD = torch.zeros_like(A), torch.zeros_like(D)
    g = s["dhy"].double()
    for t in range(T - 1, -1, -1):
        live = (t < n).double()[:, None]
        u, z, d = s["u"][t].double(), s["z"][t].double(), steps[t]
        sz = 1 / (1 + torch.exp(-z))
        dy = s["dy"][t].double() * live
        do = dy * z * sz
        dz[t] = dy * os[t] * (sz + z * sz * (1 - sz))
        a = torch.exp(d[..., None] * A)
        now = before[t] * a
        after = now.view(B, G, -1, N) + (d * u).view(B, G, -1, 1) * at(s["Bm"], t)
        dCm[t] = (do.view(B, G, -1, 1) * after).sum(2).view(B, G * N)
        g = g + (do.view(B, G, -1, 1) * at(s["Cm"], t)).view(B, E, N)
        dBm[t] = (g.view(B, G, -1, N) * (d * u).view(B, G, -1, 1)).sum(2).view(B, G * N)
        gb = (g.view(B, G, -1, N) * at(s["Bm"], t)).sum(3).view(B, E)
        du[t] = d * gb + do * D
        dD += (do * u).sum(0)
        dA += (g * now * d[..., None]).sum(0)
        pre = s["delta"][t].double() + s["delta_bias"].double()
        ddelta[t] = ((g * now * A).sum(2) + gb * u) / (1 + torch.exp(-pre)) * live
        g = g * a
    out.update(du=du, ddelta=ddelta, dA=dA, dBm=dBm, dCm=dCm, dD=dD, dz=dz, ddelta_bias=ddelta.sum((0, 1)), dh0=g)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "conv": _exact_conv, "ssm": _exact_ssm}[case["op"]](s)
