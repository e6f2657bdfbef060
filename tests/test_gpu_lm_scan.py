"""Gated linear recurrence on the GPU against its float64 definition.

Tolerance: with u = 2^-24, a state's error obeys E_t = |a| E_(t-1) + K u (|a| S_(t-1) + |b|),
S the recurrence of the magnitudes: K u bounds the relative error of a coefficient (exponential,
reciprocal and products: the exponent's argument has up to |p| <= 12 roundings' worth of error) and of the
products of coefficients that join pieces of the time axis.  What is written in 16 bits adds half a step of
the value (2^-8 for bf16)."""

import sys

import numpy as np
import pytest
import torch

import layer_rnn_forward_amd as R
from oracle import lm_oracle as O

pytestmark = pytest.mark.gpu

U, K = 2.0 ** -24, 32
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def make(mode, dtype, T, B, H, dirs, lengths=None, h0=True, dhy=True, seed=0):
    rng = np.random.default_rng([seed, T, B, H, dirs])
    g = rng.normal(size=(T, B, dirs, 2, H))
    if mode == "gated":
        g[:, :, :, 0] = g[:, :, :, 0] * 1.5 + 1.0
    else:
        g[:, :, :, 0] = 1 / (1 + np.exp(-1.5 * g[:, :, :, 0] - 2))
        g[:, :, :, 1] *= 1 - g[:, :, :, 0]
    c = dict(mode=mode, dtype=dtype, T=T, B=B, H=H, dirs=dirs,
             g=torch.tensor(g.reshape(T, B, dirs * 2 * H)).to(DT[dtype]),
             dy=torch.tensor(rng.normal(size=(T, B, dirs * H))).to(DT[dtype]),
             h0=torch.tensor(rng.normal(size=(dirs, B, H))).float() if h0 else None,
             dhy=torch.tensor(rng.normal(size=(dirs, B, H))).float() if dhy else None,
             lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32))
    return c


def cuda(t):
    return None if t is None else t.cuda()


def run(c, backward=True):
    T, B, H, dirs = c["T"], c["B"], c["H"], c["dirs"]
    dt = DT[c["dtype"]]
    g, h0, n = cuda(c["g"]), cuda(c["h0"]), cuda(c["lengths"])
    nan = float("nan")
    y = torch.full((T, B, dirs * H), nan, dtype=dt, device="cuda")
    hy = torch.full((dirs, B, H), nan, device="cuda")
    ws = torch.empty(R.rnn_scan_workspace_size(T, B, H, dirs), dtype=torch.uint8, device="cuda")
    ws.fill_(0xA5)                       # whatever the workspace held before
    R.rnn_scan_forward(c["mode"], g, h0, n, y, hy, ws)
    out = {"y": y, "hy": hy}
    if backward:
        dg = torch.full_like(g, nan)
        dh0 = torch.full((dirs, B, H), nan, device="cuda")
        R.rnn_scan_backward(c["mode"], g, h0, n, cuda(c["dy"]), cuda(c["dhy"]), dg, dh0, ws)
        out |= {"dg": dg, "dh0": dh0}
    torch.cuda.synchronize()
    return out


def expected(c):
    """{name: (value, tolerance)}"""
    T, B, H, dirs, mode = c["T"], c["B"], c["H"], c["dirs"], c["mode"]
    half = HALF[c["dtype"]]
    g = c["g"].double().numpy().reshape(T, B, dirs, 2, H)
    dy = c["dy"].double().numpy().reshape(T, B, dirs, H)
    val = {k: np.zeros((T, B, dirs, H)) for k in ("y", "dp", "dq")}
    err = {k: np.zeros((T, B, dirs, H)) for k in val}
    end = {k: np.zeros((dirs, B, H)) for k in ("hy", "dh0", "ehy", "edh0")}
    z = np.zeros(H)
    for d in range(dirs):
        for b in range(B):
            n = T if c["lengths"] is None else min(max(int(c["lengths"][b]), 0), T)
            walk = list(range(n) if d == 0 else range(n - 1, -1, -1))
            h = z if c["h0"] is None else c["h0"][d, b].double().numpy()
            s, e, keep = np.abs(h), z, []
            for t in walk:
                p, q = g[t, b, d]
                a, add, cand = O._coeffs(mode, p, q)
                keep.append((a, cand, h, e))
                e = np.abs(a) * e + K * U * (np.abs(a) * s + np.abs(add))
                s = np.abs(a) * s + np.abs(add)
                h = a * h + add
                val["y"][t, b, d], err["y"][t, b, d] = h, e
            end["hy"][d, b], end["ehy"][d, b] = h, e
            dh = z if c["dhy"] is None else c["dhy"][d, b].double().numpy()
            s, e = np.abs(dh), z
            for t, (a, cand, before, eb) in zip(reversed(walk), reversed(keep)):
                e = e + K * U * (s + np.abs(dy[t, b, d]))
                s = s + np.abs(dy[t, b, d])
                dh = dh + dy[t, b, d]
                if mode == "gated":
                    na = O.sigmoid(-g[t, b, d, 0])
                    f, f2 = (before - cand) * a * na, na * (1 - cand ** 2)
                    ef = (eb + K * U * (np.abs(before) + np.abs(cand))) * a * na
                    ef2 = K * U * na
                else:
                    f, f2, ef, ef2 = before, 1.0, eb, 0.0
                val["dp"][t, b, d], val["dq"][t, b, d] = dh * f, dh * f2
                err["dp"][t, b, d] = e * np.abs(f) + np.abs(dh) * (ef + K * U * np.abs(f))
                err["dq"][t, b, d] = e * np.abs(f2) + np.abs(dh) * (ef2 + K * U * np.abs(f2))
                dh, s, e = a * dh, np.abs(a) * s, np.abs(a) * e + K * U * np.abs(a) * s
            end["dh0"][d, b], end["edh0"][d, b] = dh, e
    dg = np.stack([val["dp"], val["dq"]], 3).reshape(T, B, -1)
    edg = np.stack([err["dp"], err["dq"]], 3).reshape(T, B, -1)
    y, ey = val["y"].reshape(T, B, -1), err["y"].reshape(T, B, -1)
    # fp32 words below the smallest normal are not resolved further than that
    tiny = 2.0 ** -126
    return {"y": (y, ey + half * (np.abs(y) + ey) + tiny), "hy": (end["hy"], end["ehy"] + U * np.abs(end["hy"]) + tiny),
            "dg": (dg, edg + half * (np.abs(dg) + edg) + tiny),
            "dh0": (end["dh0"], end["edh0"] + U * np.abs(end["dh0"]) + tiny)}


def check(got, want):
    for k, v in got.items():
        x, (ref, tol) = v.double().cpu().numpy(), want[k]
        assert np.isfinite(x).all(), k
        bad = np.abs(x - ref) > tol
        assert not bad.any(), (k, int(bad.sum()), np.argwhere(bad)[:3].tolist(), float(np.abs(x - ref).max()))


SIZES = [  # T, B, H, dirs
    (1, 1, 1, 1), (1, 3, 5, 2), (2, 1, 64, 1), (15, 2, 33, 2), (16, 1, 128, 1), (17, 5, 8, 1), (63, 1, 130, 2),
    (64, 2, 96, 1), (65, 3, 7, 2), (128, 1, 256, 1), (129, 4, 40, 1), (300, 2, 80, 2), (515, 7, 35, 2), (1237, 1, 19, 1),
]


@pytest.mark.parametrize("mode", ["gated", "linear"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_forward_backward(mode, dtype, size):
    print("CASE scan", mode, dtype, size, flush=True)
    c = make(mode, dtype, *size)
    check(run(c), expected(c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,B,H,dirs,lengths", [
    (5, 4, 6, 2, [5, 0, 3, 1]), (200, 5, 40, 2, [200, 0, 64, 65, 199]), (300, 3, 128, 1, [0, 0, 0]),
    (130, 3, 16, 2, [-7, 1000, 129]), (1000, 2, 9, 2, [1, 1000])])
def test_ragged_rows(dtype, T, B, H, dirs, lengths):
    print("CASE scan ragged", dtype, T, B, H, dirs, lengths, flush=True)
    c = make("gated", dtype, T, B, H, dirs, lengths)
    want = expected(c)
    for b, n in enumerate(lengths):      # what lies past a row's end is never used
        c["g"][max(0, n):, b] = float("nan")
        c["dy"][max(0, n):, b] = float("inf")
    check(run(c), want)


@pytest.mark.parametrize("h0,dhy", [(False, False), (True, False), (False, True)])
def test_missing_states(h0, dhy):
    c = make("gated", "f32", 150, 2, 24, 2, [150, 70], h0=h0, dhy=dhy)
    check(run(c), expected(c))


def test_no_steps_and_no_rows():
    c = make("linear", "f32", 0, 2, 5, 2)
    out = run(c)
    assert torch.equal(out["hy"].cpu(), c["h0"]) and torch.equal(out["dh0"].cpu(), c["dhy"])
    run(make("linear", "bf16", 4, 0, 5, 1))
    run(make("linear", "bf16", 4, 5, 0, 1))


def test_extreme_gates():
    """Gates far out, states that underflow, and the ends of the sigmoid."""
    c = make("gated", "f32", 260, 1, 64, 1)
    p = torch.tensor([-200.0, -88.0, -30.0, 0.0, 30.0, 88.0, 200.0, float("inf"), -float("inf")])
    c["g"][:, :, :9] = p
    c["g"][:, :, 64:73] = torch.tensor([0.0, 1e-6, -1e-3, 0.2, 0.3, 9.0, 50.0, 3.0, -3.0])
    out = run(c)
    y, hy = O.scan_forward("gated", c["g"].double().numpy(), c["h0"].double().numpy(), None, 1)
    assert np.abs(out["y"].double().cpu().numpy() - y).max() < 260 * K * U * (1 + np.abs(c["h0"].numpy()).max())
    assert torch.isfinite(out["dg"]).all() and torch.isfinite(out["dh0"]).all()


def test_nan_stays_in_its_channel():
    c = make("linear", "bf16", 200, 2, 40, 1)
    c["g"][70, 1, 3] = float("nan")
    out = run(c)
    y = out["y"].float().cpu()
    assert torch.isnan(y[70:, 1, 3]).all() and not torch.isnan(y[:70, 1, 3]).any()
    y[:, 1, 3] = 0
    assert torch.isfinite(y).all()
    dg = out["dg"].float().cpu()
    dg[:, 1, 3] = dg[:, 1, 43] = 0
    assert torch.isfinite(dg).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_repeats_are_bitwise(dtype):
    c = make("gated", dtype, 1500, 3, 200, 2, [1500, 800, 0])
    a = run(c)
    for _ in range(5):
        b = run(c)
        for k in a:
            assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_misaligned_buffers(dtype):
    """Buffers that start one element past an aligned address."""
    c = make("gated", dtype, 140, 2, 64, 2)
    want = run(c)

    def shifted(t, fill=None):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        v = buf[1:].view(t.shape)
        v.copy_(t) if fill is None else v.fill_(fill)
        return v

    g, h0, dy, dhy = (shifted(c[k].cuda()) for k in ("g", "h0", "dy", "dhy"))
    y, hy = shifted(want["y"], 7), shifted(want["hy"], 7)
    dg, dh0 = shifted(want["dg"], 7), shifted(want["dh0"], 7)
    ws = torch.empty(R.rnn_scan_workspace_size(140, 2, 64, 2), dtype=torch.uint8, device="cuda")
    R.rnn_scan_forward("gated", g, h0, None, y, hy, ws)
    R.rnn_scan_backward("gated", g, h0, None, dy, dhy, dg, dh0, ws)
    for k, v in (("y", y), ("hy", hy), ("dg", dg), ("dh0", dh0)):
        assert torch.equal(v, want[k]), k


@pytest.mark.parametrize("mode", ["gated", "linear"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H", [(1, 1), (16, 800), (3, 357), (256, 130)])
def test_step(mode, dtype, B, H):
    c = make(mode, dtype, 1, B, H, 1)
    want = expected(c)
    g, h = c["g"][0].cuda(), c["h0"][0].cuda()
    y, hy = torch.empty((B, H), dtype=DT[dtype], device="cuda"), torch.empty((B, H), device="cuda")
    R.rnn_scan_step(mode, g, h, y, hy)
    check({"y": y[None], "hy": hy[None]}, want)
    R.rnn_scan_step(mode, g, h, None, h)             # in place, no y
    assert torch.equal(h, hy)
    none = make(mode, dtype, 1, B, H, 1, h0=False)
    R.rnn_scan_step(mode, none["g"][0].cuda(), None, y, hy)
    check({"y": y[None], "hy": hy[None]}, expected(none))


def test_steps_follow_the_scan():
    """A prompt by the scan, then tokens by single steps: the states of the whole scan."""
    c = make("gated", "f32", 90, 4, 50, 1)
    whole = run(c, backward=False)
    head = dict(c, T=80, g=c["g"][:80])
    hy = run(head, backward=False)["hy"]
    y = torch.empty((4, 50), device="cuda")
    want = expected(c)["y"]
    for t in range(80, 90):
        R.rnn_scan_step("gated", c["g"][t].cuda(), hy[0], y, hy[0])
        assert (np.abs(y.double().cpu().numpy() - want[0][t]) <= want[1][t]).all()
    assert torch.isfinite(whole["y"]).all()


def test_backward_twice_and_on_another_stream():
    c = make("gated", "bf16", 700, 2, 150, 2, [700, 333])
    want = run(c)
    side = torch.cuda.Stream()
    g, h0, n, dy, dhy = (cuda(c[k]) for k in ("g", "h0", "lengths", "dy", "dhy"))
    ws = torch.empty(R.rnn_scan_workspace_size(700, 2, 150, 2), dtype=torch.uint8, device="cuda")
    y, hy = torch.empty_like(want["y"]), torch.empty_like(want["hy"])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        R.rnn_scan_forward("gated", g, h0, n, y, hy, ws)
        for _ in range(3):
            dg, dh0 = torch.full_like(g, 3.0), torch.empty_like(h0)
            R.rnn_scan_backward("gated", g, h0, n, dy, dhy, dg, dh0, ws)
            side.synchronize()
            assert torch.equal(dg, want["dg"]) and torch.equal(dh0, want["dh0"])
    assert torch.equal(y, want["y"]) and torch.equal(hy, want["hy"])


def test_graph_replays():
    c = make("gated", "bf16", 900, 2, 300, 1, [900, 450])
    want = run(c)
    g, h0, n, dy, dhy = (cuda(c[k]) for k in ("g", "h0", "lengths", "dy", "dhy"))
    ws = torch.empty(R.rnn_scan_workspace_size(900, 2, 300, 1), dtype=torch.uint8, device="cuda")
    out = {k: torch.empty_like(v) for k, v in want.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        R.rnn_scan_forward("gated", g, h0, n, out["y"], out["hy"], ws)
        R.rnn_scan_backward("gated", g, h0, n, dy, dhy, out["dg"], out["dh0"], ws)
    for i in range(4):
        for v in out.values():
            v.fill_(float(i))
        (g.float() * 2).sum().item()                  # the program's own work between replays
        graph.replay()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(out[k], want[k]), (i, k)


@pytest.mark.timeout(300)
def test_offsets_past_32_bits():
    """More than 2^31 gate values: the last channels against the same channels alone."""
    T, H = 33000, 32776
    print("CASE scan past 32 bits", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(1)
    g = torch.empty((T, 1, 2 * H), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    assert g.numel() > 1 << 31
    dy = torch.empty((T, 1, H), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    y, dg = torch.empty_like(dy), torch.empty_like(g)
    hy, dh0 = torch.empty((1, 1, H), device="cuda"), torch.empty((1, 1, H), device="cuda")
    ws = torch.empty(R.rnn_scan_workspace_size(T, 1, H, 1), dtype=torch.uint8, device="cuda")
    R.rnn_scan_forward("gated", g, None, None, y, hy, ws)
    R.rnn_scan_backward("gated", g, None, None, dy, None, dg, dh0, ws)
    torch.cuda.synchronize()
    n = 40
    sg = torch.cat([g[:, :, H - n:H], g[:, :, 2 * H - n:]], 2).contiguous()
    sdy, sy, sdg = dy[:, :, H - n:].contiguous(), torch.empty((T, 1, n), dtype=torch.bfloat16, device="cuda"), None
    sdg, shy, sdh0 = torch.empty_like(sg), torch.empty((1, 1, n), device="cuda"), torch.empty((1, 1, n), device="cuda")
    sws = torch.empty(R.rnn_scan_workspace_size(T, 1, n, 1), dtype=torch.uint8, device="cuda")
    R.rnn_scan_forward("gated", sg, None, None, sy, shy, sws)
    R.rnn_scan_backward("gated", sg, None, None, sdy, None, sdg, sdh0, sws)
    # both are roundings of the same values: at most one bf16 step (two halves) apart
    both = [(y[:, :, H - n:], sy), (dg[:, :, H - n:H], sdg[:, :, :n]), (dg[:, :, 2 * H - n:], sdg[:, :, n:])]
    for a, b in both:
        assert ((a.float() - b.float()).abs() <= 2 * 2.0 ** -8 * b.float().abs() + 1e-5).all()
    assert ((hy[:, :, H - n:] - shy).abs() <= 1e-5).all() and ((dh0[:, :, H - n:] - sdh0).abs() <= 1e-5).all()
    sys.stdout.flush()
