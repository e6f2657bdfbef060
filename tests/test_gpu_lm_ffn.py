"""Gated feed-forward block on the GPU against its float64 definition.

Inputs are small multiples of powers of two, chosen so that the projections g and u are exact in fp32 in any
order of summation (products of 5-bit numbers, sums below 2^24 units): what is left are the roundings that
the tolerances count.  With u = 2^-24 and h = 2^-8 (bf16) or u (fp32), half a step of a value:
 * the activation's fp32 error: 64 u (|a| + |g|);
 * the gated product is held in the element type: h |a u|;
 * RNN_SAVE_FULL holds act(g) and u act'(g) in bf16 mode as 14 bits with a shared exponent for 32 values: 2^-14
   of the row's largest magnitude;
 * dgate and dup are held in the element type;
 * a sum of n products in fp32: n u times the sum of the magnitudes;
 * each output: h of itself.
Where the sums are long enough for roundings to be independent, the bf16 outputs' norms are also held to two
half steps."""

import numpy as np
import pytest
import torch

import layer_rnn_forward_amd as R
from oracle import lm_oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": U, "bf16": 2.0 ** -8}


def make(M, D, F, dtype, seed=0):
    rng = np.random.default_rng([seed, M, D, F])

    def grid(shape, unit):
        return np.clip(np.rint(rng.normal(size=shape) * 5), -15, 15) * unit

    near = 2.0 ** -np.round(np.log2(max(D, 1)) / 2)
    return dict(M=M, D=D, F=F, dtype=dtype, x=grid((M, D), 2.0 ** -2), w_in=grid((2 * F, D), near * 2.0 ** -2),
                w_out=grid((D, F), 2.0 ** -np.round(np.log2(max(F, 1)) / 2) * 2.0 ** -2), dy=grid((M, D), 2.0 ** -2))


def dev(c, k):
    return torch.tensor(c[k]).to(DT[c["dtype"]]).cuda()


def run(c, act, save, want_grads=("dx", "dw_in", "dw_out")):
    M, D, F, dtype = c["M"], c["D"], c["F"], c["dtype"]
    x, w_in, w_out, dy = (dev(c, k) for k in ("x", "w_in", "w_out", "dy"))
    nan = float("nan")
    ws = torch.full((R.rnn_ffn_workspace_size(M, D, F, dtype, save),), 0xFF, dtype=torch.uint8, device="cuda")
    reserve = torch.full((R.rnn_ffn_reserve_size(M, D, F, dtype, save),), 0xFF, dtype=torch.uint8, device="cuda")
    y = torch.full_like(x, nan)
    R.rnn_ffn_forward(act, x, w_in, w_out, y, ws, save, reserve)
    out = {"y": y}
    if save != "none":
        ws.fill_(0xFF)                                 # backward reads the reserve, not the workspace
        kept = reserve.clone()
        g = {k: torch.full_like(v, nan) if k in want_grads else None
             for k, v in (("dx", x), ("dw_in", w_in), ("dw_out", w_out))}
        R.rnn_ffn_backward(act, None if save == "int8" else x, w_in, w_out, dy, g["dx"], g["dw_in"], g["dw_out"], ws,
                           save, reserve)
        assert torch.equal(kept, reserve)
        out |= {k: v for k, v in g.items() if v is not None}
    torch.cuda.synchronize()
    return out


def expected(c, act, save):
    """{name: (value, tolerance)}"""
    x, w_in, w_out, dy, F = c["x"], c["w_in"], c["w_out"], c["dy"], c["F"]
    half = HALF[c["dtype"]]
    gu = x @ w_in.T
    g, u = gu[:, :F], gu[:, F:]
    a, _ = O.act_pair(act, g)
    ea = 64 * U * (np.abs(a) + np.abs(g))
    h = a * u
    eh = ea * np.abs(u) + half * np.abs(h)

    def product(p, ep, w, n):
        v = p @ w
        e = ep @ np.abs(w) + n * U * (np.abs(p) @ np.abs(w))
        return v, e + half * (np.abs(v) + e)

    out = {"y": product(h, eh, w_out.T, F)}
    if save == "none":
        return out
    if save == "int8":
        x, g, u = O.checkpoint_round(x), O.checkpoint_round(g), O.checkpoint_round(u)
    a, da = O.act_pair(act, g)
    ea = 64 * U * (np.abs(a) + np.abs(g))
    h = a * u
    eh = ea * np.abs(u) + half * np.abs(h)
    p = u * da
    ep = 64 * U * (1 + np.abs(g)) * np.abs(u)
    if save == "full" and c["dtype"] == "bf16" and g.size:
        ea = ea + 2.0 ** -14 * np.abs(a).max(1, keepdims=True)
        ep = ep + 2.0 ** -14 * np.abs(p).max(1, keepdims=True)
    dh = dy @ w_out
    edh = c["D"] * U * (np.abs(dy) @ np.abs(w_out))
    dg, du = dh * p, dh * a
    edg = edh * (np.abs(p) + ep) + np.abs(dh) * ep
    edu = edh * (np.abs(a) + ea) + np.abs(dh) * ea
    edg, edu = edg + half * (np.abs(dg) + edg), edu + half * (np.abs(du) + edu)
    dgu, edgu = np.concatenate([dg, du], 1), np.concatenate([edg, edu], 1)
    out["dx"] = product(dgu, edgu, w_in, 2 * F)
    v, e = product(x.T, np.zeros_like(x.T), dgu, c["M"])
    e = e + (np.abs(x).T @ edgu) * (1 + half)
    out["dw_in"] = v.T, e.T
    v, e = product(dy.T, np.zeros_like(dy.T), h, c["M"])
    out["dw_out"] = v, e + (np.abs(dy).T @ eh) * (1 + half)
    return out


def check(got, want, c):
    for k, v in got.items():
        x, (ref, tol) = v.double().cpu().numpy(), want[k]
        assert np.isfinite(x).all(), k
        bad = np.abs(x - ref) > tol + 1e-30
        assert not bad.any(), (k, int(bad.sum()), np.argwhere(bad)[:3].tolist(), float(np.abs(x - ref).max()))
        if c["dtype"] == "bf16" and min(c["M"], c["D"], c["F"]) >= 64:
            assert np.linalg.norm(x - ref) <= 2 * 2.0 ** -8 * np.linalg.norm(ref), k


SIZES = [  # M, D, F
    (1, 1, 1), (1, 8, 8), (2, 5, 3), (3, 64, 64), (16, 200, 72), (17, 72, 200), (33, 40, 9), (64, 64, 64), (100, 96, 33),
    (130, 130, 70), (257, 264, 136), (128, 256, 512), (300, 357, 129), (513, 64, 1021), (40, 1000, 48), (700, 160, 320),
    (260, 8, 300), (16, 2048, 512), (9, 504, 1000), (384, 320, 640),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("act,save", [("silu", "none"), ("silu", "full"), ("gelu", "int8"), ("sigmoid", "full")])
def test_forward_backward(dtype, size, act, save):
    print("CASE ffn", dtype, size, act, save, flush=True)
    c = make(*size, dtype)
    check(run(c, act, save), expected(c, act, save), c)


@pytest.mark.parametrize("M", range(1, 20))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_few_rows(M, dtype):
    print("CASE ffn rows", M, dtype, flush=True)
    for D, F in ((320, 416), (63, 130)):
        c = make(M, D, F, dtype, seed=2)
        check(run(c, "gelu", "none"), expected(c, "gelu", "none"), c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("save", ["full", "int8"])
def test_each_gradient_alone(dtype, save):
    c = make(90, 72, 56, dtype)
    every = run(c, "silu", save)
    for k in ("dx", "dw_in", "dw_out"):
        one = run(c, "silu", save, (k,))
        assert torch.equal(one[k], every[k]), k


def test_no_rows():
    c = make(0, 24, 40, "bf16")
    out = run(c, "silu", "full")
    assert (out["dw_in"] == 0).all() and (out["dw_out"] == 0).all() and out["y"].shape == (0, 24)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("save", ["full", "int8"])
def test_repeats_are_bitwise(dtype, save):
    c = make(300, 264, 392, dtype)
    a = run(c, "gelu", save)
    for _ in range(3):
        b = run(c, "gelu", save)
        for k in a:
            assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("M", [4, 150])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_misaligned_tensors(M, dtype):
    """Tensors that start one element past an aligned address."""
    D, F, save = 64, 96, "full"
    c = make(M, D, F, dtype)
    want = run(c, "silu", save)

    def shifted(t):
        buf = torch.full((t.numel() + 1,), 5.0, dtype=t.dtype, device="cuda")
        v = buf[1:].view(t.shape)
        v.copy_(t)
        return v

    x, w_in, w_out, dy = (shifted(dev(c, k)) for k in ("x", "w_in", "w_out", "dy"))
    y, dx, dwi, dwo = (shifted(torch.zeros_like(t)) for t in (x, x, w_in, w_out))
    ws = torch.empty(R.rnn_ffn_workspace_size(M, D, F, dtype, save), dtype=torch.uint8, device="cuda")
    reserve = torch.empty(R.rnn_ffn_reserve_size(M, D, F, dtype, save), dtype=torch.uint8, device="cuda")
    R.rnn_ffn_forward("silu", x, w_in, w_out, y, ws, save, reserve)
    R.rnn_ffn_backward("silu", x, w_in, w_out, dy, dx, dwi, dwo, ws, save, reserve)
    for k, v in (("y", y), ("dx", dx), ("dw_in", dwi), ("dw_out", dwo)):
        assert torch.equal(v, want[k]), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_row_of_infinities_stays_in_its_row(dtype):
    c = make(140, 72, 80, dtype)
    clean = run(c, "silu", "full")
    x, w_in, w_out, dy = (dev(c, k) for k in ("x", "w_in", "w_out", "dy"))
    x[70] = float("inf")
    ws = torch.empty(R.rnn_ffn_workspace_size(140, 72, 80, dtype, "full"), dtype=torch.uint8, device="cuda")
    reserve = torch.empty(R.rnn_ffn_reserve_size(140, 72, 80, dtype, "full"), dtype=torch.uint8, device="cuda")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    R.rnn_ffn_forward("silu", x, w_in, w_out, y, ws, "full", reserve)
    R.rnn_ffn_backward("silu", x, w_in, w_out, dy, dx, None, None, ws, "full", reserve)
    rows = [i for i in range(140) if i != 70]
    assert torch.equal(y[rows], clean["y"][rows]) and torch.equal(dx[rows], clean["dx"][rows])
    assert not torch.isfinite(y[70]).any() and not torch.isfinite(dx[70]).any()


def test_graph_and_stream():
    c = make(200, 136, 264, "bf16")
    want = run(c, "silu", "int8")
    x, w_in, w_out, dy = (dev(c, k) for k in ("x", "w_in", "w_out", "dy"))
    ws = torch.empty(R.rnn_ffn_workspace_size(200, 136, 264, "bf16", "int8"), dtype=torch.uint8, device="cuda")
    reserve = torch.empty(R.rnn_ffn_reserve_size(200, 136, 264, "bf16", "int8"), dtype=torch.uint8, device="cuda")
    out = {k: torch.empty_like(v) for k, v in want.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        R.rnn_ffn_forward("silu", x, w_in, w_out, out["y"], ws, "int8", reserve)
        R.rnn_ffn_backward("silu", None, w_in, w_out, dy, out["dx"], out["dw_in"], out["dw_out"], ws, "int8", reserve)
    for i in range(3):
        for v in out.values():
            v.fill_(float(i))
        (x.float() * 2).sum().item()
        graph.replay()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(out[k], want[k]), (i, k)
