"""The operators at the sizes where they take other paths: each tile of the feed-forward products, k split among
workgroups, few rows on both sides of their limits; sequences over many groups of chunks, steps that grow.

Tolerances as in the operators' own tests (derived there); a product whose k is split adds the same number of
products in another order, which the bound on n products covers."""

import numpy as np
import pytest
import torch

import layer_rnn_forward_amd as R
from tests import test_gpu_lm_ffn as ffn
from tests import test_gpu_lm_scan as scan

pytestmark = pytest.mark.gpu


@pytest.mark.timeout(300)
@pytest.mark.parametrize("size", [(8190, 500, 2030), (4085, 1000, 2030), (8190, 2040, 130)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("act,save", [("silu", "full"), ("gelu", "int8")])
def test_large_tiles(size, act, save):
    print("CASE ffn large", size, act, save, flush=True)
    c = ffn.make(*size, "bf16")
    ffn.check(ffn.run(c, act, save), ffn.expected(c, act, save), c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(5000, 40, 24), (130, 130, 2500), (3000, 72, 56), (70, 33, 5001), (1111, 200, 7)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("act,save", [("silu", "full"), ("sigmoid", "int8")])
def test_split_products(dtype, size, act, save):
    print("CASE ffn split", dtype, size, act, save, flush=True)
    c = ffn.make(*size, dtype)
    got = ffn.run(c, act, save)
    ffn.check(got, ffn.expected(c, act, save), c)
    again = ffn.run(c, act, save)
    for k in got:
        assert torch.equal(got[k], again[k]), k
    for k in ("dx", "dw_in", "dw_out"):
        assert torch.equal(ffn.run(c, act, save, (k,))[k], got[k]), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [(70, 2501, 130), (130, 1500, 24), (257, 5000, 72), (300, 4100, 700), (256, 4000, 2048), (90, 700, 1)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("act,save", [("gelu", "none"), ("silu", "full"), ("sigmoid", "int8")])
def test_split_projections(dtype, size, act, save):
    print("CASE ffn split projections", dtype, size, act, save, flush=True)
    c = ffn.make(*size, dtype)
    got = ffn.run(c, act, save)
    ffn.check(got, ffn.expected(c, act, save), c)
    again = ffn.run(c, act, save)
    for k in got:
        assert torch.equal(got[k], again[k]), k


@pytest.mark.parametrize("M", [8, 9, 16, 17, 32, 33, 63, 64, 65])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_on_both_sides_of_a_limit(M, dtype):
    print("CASE ffn limits", M, dtype, flush=True)
    for D, F in ((8, 16), (96, 264), (520, 1000), (33, 31), (1030, 17)):
        c = ffn.make(M, D, F, dtype, seed=3)
        ffn.check(ffn.run(c, "silu", "none"), ffn.expected(c, "silu", "none"), c)


def test_few_rows_add_no_rounding():
    """bf16, up to 64 rows: the gated product is passed on in 16 bits, so the output is off by its own rounding
    (half a step) and 2^-16 of the magnitudes summed."""
    for M, D, F in ((1, 256, 2048), (7, 100, 999), (40, 64, 640)):
        c = ffn.make(M, D, F, "bf16", seed=4)
        y = ffn.run(c, "silu", "none")["y"].double().cpu().numpy()
        gu = c["x"] @ c["w_in"].T
        g, u = gu[:, :F], gu[:, F:]
        a, _ = ffn.O.act_pair("silu", g)
        h = a * u
        ref = h @ c["w_out"].T
        mags = np.abs(h) @ np.abs(c["w_out"]).T
        e = (2.0 ** -16 + F * ffn.U) * mags + 64 * ffn.U * ((np.abs(a) + np.abs(g)) * np.abs(u)) @ np.abs(c["w_out"]).T
        assert (np.abs(y - ref) <= e + 2.0 ** -8 * (np.abs(ref) + e) + 1e-30).all(), (M, D, F)


@pytest.mark.parametrize("M", [3, 200])
def test_rows_of_infinities_without_saving(M):
    c = ffn.make(M, 72, 80, "bf16")
    clean = ffn.run(c, "silu", "none")["y"]
    x, w_in, w_out = (ffn.dev(c, k) for k in ("x", "w_in", "w_out"))
    x[1] = float("inf")
    y = torch.empty_like(x)
    ws = torch.empty(R.rnn_ffn_workspace_size(M, 72, 80, "bf16", "none"), dtype=torch.uint8, device="cuda")
    R.rnn_ffn_forward("silu", x, w_in, w_out, y, ws)
    rows = [i for i in range(M) if i != 1]
    assert torch.equal(y[rows], clean[rows]) and not torch.isfinite(y[1]).any()


@pytest.mark.parametrize("act", ["sigmoid", "silu", "gelu"])
@pytest.mark.parametrize("M", [2, 100])
def test_large_projections(act, M):
    """Projections far out: activations saturate, and nothing overflows on the way."""
    D, F = 8, 8
    x = torch.zeros(M, D, device="cuda")
    x[:, 0] = 1
    w_in, w_out = torch.zeros(2 * F, D, device="cuda"), torch.eye(D, F, device="cuda")
    g = torch.tensor([-1e30, -300.0, -90.0, -20.0, 20.0, 90.0, 300.0, 1e8], device="cuda")
    w_in[:F, 0], w_in[F:, 0] = g, 1
    y, dx = torch.empty_like(x), torch.empty_like(x)
    ws = torch.empty(R.rnn_ffn_workspace_size(M, D, F, "f32", "full"), dtype=torch.uint8, device="cuda")
    reserve = torch.empty(R.rnn_ffn_reserve_size(M, D, F, "f32", "full"), dtype=torch.uint8, device="cuda")
    want = ffn.O.act_pair(act, g.double().cpu().numpy().clip(-1e10, None))[0]
    want = np.where(np.arange(8) == 0, 0.0, want)       # all three vanish there
    for save in ("none", "full"):
        R.rnn_ffn_forward(act, x, w_in, w_out, y, ws, save, reserve)
        got = y.double().cpu().numpy()
        assert (np.abs(got - want) <= 200 * ffn.U * np.abs(want) + 1e-30).all(), save
    R.rnn_ffn_backward(act, x, w_in, w_out, torch.ones_like(y), dx, None, None, ws, "full", reserve)
    assert torch.isfinite(dx).all()


@pytest.mark.parametrize("mode", ["gated", "linear"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scan_over_many_groups(mode, dtype):
    """More chunks than two groups hold, in both passes and both directions, with rows that end anywhere."""
    T = 4500
    print("CASE scan groups", mode, dtype, flush=True)
    c = scan.make(mode, dtype, T, 3, 70, 2, [T, 1023, 1024])
    scan.check(scan.run(c), scan.expected(c))


def test_linear_steps_that_grow_from_zero():
    """|a| > 1 over many steps: the product of a piece's coefficients overflows, but a state of zero stays zero
    until something is added."""
    T, H = 700, 64
    g = torch.zeros(T, 1, 2 * H)
    g[:, :, :H] = 1e30
    g[-1, :, H:] = 1.0
    y, hy = torch.empty(T, 1, H, device="cuda"), torch.empty(1, 1, H, device="cuda")
    ws = torch.empty(R.rnn_scan_workspace_size(T, 1, H, 1), dtype=torch.uint8, device="cuda")
    R.rnn_scan_forward("linear", g.cuda(), None, None, y, hy, ws)
    assert (y[:-1] == 0).all() and (y[-1] == 1).all() and (hy == 1).all()


def test_expired_waits_are_not_reported_after_a_pass():
    c = scan.make("gated", "bf16", 3000, 1, 256, 1)
    g, h0 = c["g"].cuda(), c["h0"].cuda()
    ws = torch.full((R.rnn_scan_workspace_size(3000, 1, 256, 1),), 0xFF, dtype=torch.uint8, device="cuda")
    y, hy = torch.empty(3000, 1, 256, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 1, 256, device="cuda")
    for t in (3000, 100):                               # several chunks, one chunk
        ws.fill_(0xFF)
        R.rnn_scan_forward("gated", g[:t], h0, None, y[:t], hy, ws)
        assert ws[:4].view(torch.int32).item() == 0


def test_binding_refuses_tensors_of_other_shapes_and_types():
    x = torch.zeros(4, 8, device="cuda")
    ws = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="shape"):
        R.rnn_ffn_forward("silu", x, torch.zeros(30, 8, device="cuda"), torch.zeros(8, 16, device="cuda"), x, ws)
    with pytest.raises(ValueError, match="float32"):
        R.rnn_ffn_forward("silu", x, torch.zeros(32, 8, device="cuda", dtype=torch.bfloat16), torch.zeros(8, 16, device="cuda"), x, ws)
    with pytest.raises(ValueError, match="contiguous"):
        R.rnn_ffn_forward("silu", torch.zeros(8, 4, device="cuda").t(), torch.zeros(32, 8, device="cuda"),
                          torch.zeros(8, 16, device="cuda"), x, ws)
    with pytest.raises(ValueError, match="device"):
        R.rnn_ffn_forward("silu", x, torch.zeros(32, 8), torch.zeros(8, 16, device="cuda"), x, ws)
    with pytest.raises(R.RNNError):
        R.rnn_ffn_forward("silu", x, torch.zeros(32, 8, device="cuda"), torch.zeros(8, 16, device="cuda"), x, ws[:256])
    with pytest.raises(R.RNNError):
        R.rnn_checkpoint_store(x, ws[:7])
    with pytest.raises(ValueError, match="C int"):
        R.rnn_scan_workspace_size(1 << 32, 1, 1)


@pytest.mark.parametrize("dtype,T,B,H,dirs", [("bf16", 3000, 2, 200, 2), ("f32", 700, 3, 75, 1), ("bf16", 100, 2, 64, 1)])
def test_backward_again_and_again(dtype, T, B, H, dirs):
    """Backward passes that follow one forward pass, eager or in a graph of their own, give the same gradients."""
    c = scan.make("gated", dtype, T, B, H, dirs, [T] + [T // 3] * (B - 1))
    want = scan.run(c)
    g, h0, n, dy, dhy = (scan.cuda(c[k]) for k in ("g", "h0", "lengths", "dy", "dhy"))
    ws = torch.full((R.rnn_scan_workspace_size(T, B, H, dirs),), 0x11, dtype=torch.uint8, device="cuda")
    R.rnn_scan_forward("gated", g, h0, n, torch.empty_like(want["y"]), torch.empty_like(want["hy"]), ws)
    dg, dh0 = torch.empty_like(g), torch.empty_like(h0)
    for _ in range(3):
        dg.fill_(3.0)
        R.rnn_scan_backward("gated", g, h0, n, dy, dhy, dg, dh0, ws)
        assert torch.equal(dg, want["dg"]) and torch.equal(dh0, want["dh0"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        R.rnn_scan_backward("gated", g, h0, n, dy, dhy, dg, dh0, ws)
    for _ in range(3):
        dg.fill_(5.0)
        (g.float() * 2).sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dg, want["dg"]) and torch.equal(dh0, want["dh0"])
