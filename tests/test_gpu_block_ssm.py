"""Selective state-space scan on the GPU against the definition in 64 bits; tolerances are the oracle's bounds on an
evaluation in fp32 and half a step of the output's type."""

import numpy as np
import pytest
import torch

import layer_rnn_forward_amd as R
from oracle.bounds import Bound, check
from tests.block_gpu import INPUTS, gpu, room, ssm_case, ssm_run, ssm_want

pytestmark = pytest.mark.gpu
FP32 = ("hy", "dA", "dD", "ddelta_bias", "dh0")


def compare(mode, c, dtype, wide=0, backward=True):
    got, want = ssm_run(mode, c, wide, backward), ssm_want(mode, c, backward)
    assert set(got) == set(want)
    for k, v in want.items():
        check(k, got[k], v, "f32" if k in FP32 else dtype)
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,B,E,N,G", [(1, 1, 1, 1, 1), (3, 2, 5, 4, 1), (5, 2, 16, 16, 1), (64, 1, 17, 16, 1), (65, 2, 33, 16, 1), (130, 2, 20, 8, 1),
                                       (100, 1, 70, 3, 1), (40, 2, 24, 13, 3), (70, 3, 12, 32, 2), (66, 1, 9, 64, 1), (63, 2, 40, 5, 4),
                                       (200, 1, 64, 16, 2), (50, 1, 8, 41, 1)])
def test_sequences(dtype, T, B, E, N, G):
    print("CASE ssm", dtype, T, B, E, N, G, flush=True)
    compare("softplus", ssm_case(T, B, E, N, G, dtype), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [2, 7, 16, 30, 50])
def test_steps_as_given(dtype, N):
    """Linear d, without the gate, and without bias and skip."""
    compare("linear", ssm_case(90, 2, 19, N, 1, dtype, mode="linear"), dtype)
    compare("linear", ssm_case(70, 2, 19, N, 1, dtype, mode="linear", gated=False), dtype)
    compare("softplus", ssm_case(70, 2, 18, N, 2, dtype, extras=False, state=False), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,lengths", [(70, [70, 0, 1, 64]), (200, [128, 63, 200, 65]), (40, [-3, 99, 17, 40])])
@pytest.mark.parametrize("N", [4, 16, 40])
def test_ragged_rows(dtype, T, lengths, N):
    """Lengths within, below and above the range; what lies past a row's length is not used."""
    c = ssm_case(T, 4, 18, N, 1, dtype, lengths)
    got = compare("softplus", c, dtype)
    for b, n in enumerate(lengths):
        for k in ("u", "delta", "z", "Bm", "Cm", "dy"):
            c[k][max(n, 0):, b] = float("nan") if b % 2 else float("inf")
    again = ssm_run("softplus", c)
    for k in got:
        assert torch.equal(got[k], again[k]), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B", [1, 2])
def test_slices_of_wider_tensors(dtype, B):
    for T in (1, 70):
        c = ssm_case(T, B, 21, 16, 1, dtype)
        got, want = compare("softplus", c, dtype, wide=11), ssm_run("softplus", c)
        for k in want:
            assert torch.equal(got[k], want[k]), k


@pytest.mark.parametrize("N", [2, 16, 40])
def test_one_step_in_rows_far_apart(N):
    """A step's rows 2^27 elements apart (the last step of sequences that lie one after the other): B * ld is past what
    several steps may have, and a lane's offset of three steps past 32 bits."""
    c = ssm_case(1, 4, 21, N, 1, "f32")
    want = ssm_run("softplus", c)
    ld, at = 1 << 27, 0
    store = torch.empty(3 * ld + 1024, device="cuda")

    def far(t):
        nonlocal at
        v = store[at:].as_strided(t.shape, (4 * ld, ld, 1))
        at += t.shape[-1]
        return v.copy_(t)
    g = {k: far(v) if k in ("u", "delta", "Bm", "Cm", "z", "dy") else gpu(v) for k, v in c.items()}
    got = {k: far(torch.full(v.shape, 7.0)) if k in ("y", "du", "ddelta", "dBm", "dCm", "dz") else torch.full_like(v, 7.0)
           for k, v in want.items()}
    assert at <= 1024
    ws = room(R.rnn_ssm_workspace_size(1, 4, 21, N, 1, "full"))
    R.rnn_ssm_forward("softplus", *(g[k] for k in INPUTS), g["h0"], None, got["y"], got["hy"], ws, "full")
    R.rnn_ssm_backward("softplus", *(g[k] for k in INPUTS), g["h0"], None, g["dy"], g["dhy"], got["du"], got["ddelta"],
                       got["dA"], got["dBm"], got["dCm"], got["dD"], got["dz"], got["ddelta_bias"], got["dh0"], ws)
    for k in want:
        assert torch.equal(got[k], want[k]), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_channels(dtype):
    """B and C of no channels: their gradients are 0."""
    c = ssm_case(9, 2, 6, 8, 2, dtype)
    for k in ("u", "delta", "z", "dy"):
        c[k] = c[k][..., :0].contiguous()
    c |= {"A": c["A"][:0], "D": c["D"][:0], "delta_bias": c["delta_bias"][:0], "h0": c["h0"][:, :0].contiguous(),
          "dhy": c["dhy"][:, :0].contiguous()}
    got = ssm_run("softplus", c)
    assert (got["dBm"] == 0).all() and (got["dCm"] == 0).all() and got["dBm"].shape == (9, 2, 16)


def test_no_steps():
    c = ssm_case(0, 2, 10, 16, 1, "f32")
    got = compare("softplus", c, "f32")
    assert torch.equal(got["hy"].cpu(), c["h0"]) and torch.equal(got["dh0"].cpu(), c["dhy"])


def test_inference_is_trainings_forward():
    c = ssm_case(150, 3, 50, 16, 1, "bf16", [150, 20, 77])
    a, b = ssm_run("softplus", c), ssm_run("softplus", c, backward=False)
    assert torch.equal(a["y"], b["y"]) and torch.equal(a["hy"], b["hy"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,G", [(3, 1), (8, 2), (16, 1), (29, 1), (64, 2)])
def test_single_steps(dtype, N, G):
    """Every step by itself, the state updated in place, against the definition of the sequence."""
    c = ssm_case(40, 3, 22, N, G, dtype)
    want = ssm_want("softplus", c, backward=False)
    g = {k: gpu(v) for k, v in c.items()}
    h, y = g["h0"].clone(), torch.empty_like(g["u"])
    for t in range(40):
        at = [g[k] if k in ("A", "D", "delta_bias") else g[k][t] for k in INPUTS]
        R.rnn_ssm_step("softplus", *at, h, y[t], h)
    check("y", y, want["y"], dtype)
    check("hy", h, want["hy"])


def test_states_carried_in_place():
    """A sequence in pieces, hy over h0; gradients with dh0 over dhy."""
    c = ssm_case(150, 2, 40, 16, 1, "f32")
    want = ssm_want("softplus", c)
    g = {k: gpu(v) for k, v in c.items()}
    h, y = g["h0"].clone(), torch.empty_like(g["u"])
    ws = room(R.rnn_ssm_workspace_size(150, 2, 40, 16, 1))
    for a, b in ((0, 70), (70, 71), (71, 150)):
        at = [g[k] if k in ("A", "D", "delta_bias") else g[k][a:b] for k in INPUTS]
        R.rnn_ssm_forward("softplus", *at, h, None, y[a:b], h, ws)
    check("y", y, want["y"])
    check("hy", h, want["hy"])
    ws = room(R.rnn_ssm_workspace_size(150, 2, 40, 16, 1, "full"))
    R.rnn_ssm_forward("softplus", *(g[k] for k in INPUTS), g["h0"], None, y, None, ws, "full")
    d = g["dhy"].clone()
    R.rnn_ssm_backward("softplus", *(g[k] for k in INPUTS), g["h0"], None, g["dy"], d, *[None] * 8, d, ws)
    check("dh0", d, want["dh0"])


def test_not_wanted_gradients():
    c = ssm_case(80, 2, 30, 16, 1, "bf16")
    want = ssm_run("softplus", c)
    g = {k: gpu(v) for k, v in c.items()}
    y, ws = torch.empty_like(g["u"]), room(R.rnn_ssm_workspace_size(80, 2, 30, 16, 1, "full"))
    R.rnn_ssm_forward("softplus", *(g[k] for k in INPUTS), g["h0"], None, y, None, ws, "full")
    names = ("du", "ddelta", "dA", "dBm", "dCm", "dD", "dz", "ddelta_bias", "dh0")
    for name in names:
        out = [torch.empty_like(want[k]) if k == name else None for k in names]
        R.rnn_ssm_backward("softplus", *(g[k] for k in INPUTS), g["h0"], None, g["dy"], g["dhy"], *out, ws)
        assert torch.equal(out[names.index(name)], want[name]), name


def test_strong_decay_and_large_states():
    """Decays far below fp32's range: a state of 1e30 that the steps carry down to the inputs' size, and resets."""
    c = ssm_case(96, 1, 16, 4, 1, "f32", seed=5, mode="linear", gated=False, extras=False)
    c["A"][:] = torch.tensor([-1.0, -40.0, -0.001, -700.0])
    c["delta"][:] = 1.0
    c["h0"][:] = 1e30
    c["dhy"][:] = 1e-30
    compare("linear", c, "f32")
    c["delta"][20:28] = 30.0
    compare("linear", c, "f32")


def test_large_and_small_deltas():
    """softplus at both ends: e^x far below 0, x far above."""
    c = ssm_case(70, 2, 20, 16, 1, "f32", seed=6)
    c["delta"][:20] = -60.0
    c["delta"][20:30] = -100.0
    c["delta"][30:40] = 40.0
    compare("softplus", c, "f32")


def test_no_rows():
    c = ssm_case(5, 0, 6, 4, 1, "f32")
    got = ssm_run("softplus", c)
    for k in ("dA", "dD", "ddelta_bias"):
        assert not got[k].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,lengths", [(16, None), (16, [700, 300]), (3, [5, 700]), (40, [700, 0])])
def test_segments(dtype, N, lengths):
    """Few channels and many steps: the time axis in segments, rows that end in the first ones."""
    compare("softplus", ssm_case(700, 2, 20, N, 1, dtype, lengths, seed=3), dtype)


@pytest.mark.parametrize("N", [2, 16])
def test_parts_of_segments(N):
    """So many channels that backward's segments are cut into parts for the first launch."""
    compare("softplus", ssm_case(200, 2, 500, N, 500, "f32", [200, 150], seed=4), "f32")


def test_segments_in_place():
    """hy over h0 and dh0 over dhy where the first segment reads what the last one writes, and the other way round."""
    c = ssm_case(600, 1, 24, 16, 1, "f32", seed=8)
    want = ssm_run("softplus", c)
    g = {k: gpu(v) for k, v in c.items()}
    h, y, ws = g["h0"].clone(), torch.empty_like(g["u"]), room(R.rnn_ssm_workspace_size(600, 1, 24, 16, 1, "full"))
    R.rnn_ssm_forward("softplus", *(g[k] for k in INPUTS), h, None, y, h, ws, "full")
    assert torch.equal(h, want["hy"]) and torch.equal(y, want["y"])
    d = g["dhy"].clone()
    R.rnn_ssm_backward("softplus", *(g[k] for k in INPUTS), g["h0"], None, g["dy"], d, *[None] * 8, d, ws)
    assert torch.equal(d, want["dh0"])


def test_strong_decay_over_segments():
    """A state of 1e30 carried through segments whose decay is far below fp32's range."""
    c = ssm_case(640, 1, 16, 4, 1, "f32", seed=5, mode="linear", gated=False, extras=False)
    c["A"][:] = torch.tensor([-0.2, -1.0, -1e-3, 0.0])
    c["delta"][:] = 1.0
    c["u"] *= 1e-20
    c["h0"][:] = 1e30
    c["dhy"][:] = 1e-30
    compare("linear", c, "f32")


def test_growing_states():
    """Positive A: states that grow by e^40, and one that starts at zero beside them."""
    c = ssm_case(400, 1, 8, 4, 1, "f32", seed=9, mode="linear", gated=False, extras=False)
    c["A"][:] = torch.tensor([0.1, 0.05, 0.0, -0.1])
    c["delta"][:] = 1.0
    c["h0"][:, ::2] = 0.0
    c["u"][:, :, ::2] = 0.0
    compare("linear", c, "f32")


def test_infinite_values_stay_in_their_row():
    """An infinite input or a NaN state touches its own row and channel only."""
    c = ssm_case(70, 3, 20, 16, 1, "f32", seed=10)
    want = ssm_run("softplus", c)
    c["u"][30, 1, 4] = float("inf")
    c["h0"][2, 7, 3] = float("nan")
    got = ssm_run("softplus", c)
    assert torch.equal(got["y"][:, 0], want["y"][:, 0]) and torch.equal(got["hy"][0], want["hy"][0])
    assert torch.equal(got["y"][:30, 1], want["y"][:30, 1]) and not got["y"][31:, 1, 4].isfinite().any()
    others = [e for e in range(20) if e != 7]
    assert torch.equal(got["y"][:, 2][:, others], want["y"][:, 2][:, others]) and got["hy"][2, 7].isnan()[3]
    for k in ("du", "ddelta", "dz"):
        assert torch.equal(got[k][:, 0], want[k][:, 0])


def test_infinite_coefficient_reaches_only_its_own_sums():
    """A tile with lanes to spare: an infinite C must not make the sums over channels NaN through them."""
    c = ssm_case(20, 1, 5, 16, 1, "f32", seed=11, gated=False)
    c["Cm"][7, 0, 3] = float("inf")
    c["dy"][7] = c["dy"][7].abs() + 0.1
    c["u"] = c["u"].abs() + 0.1
    got = ssm_run("softplus", c)
    assert (got["dBm"][:8, 0, 3] == float("inf")).all() and got["dBm"][8:, 0, 3].isfinite().all()
    assert got["dBm"][:, 0, [n for n in range(16) if n != 3]].isfinite().all() and got["dCm"].isfinite().all()


def positive(T, N, dtype, seed):
    """Inputs whose products and sums cannot cancel: what is infinite stays so, with its sign."""
    c = ssm_case(T, 3, 20, N, 1, dtype, seed=seed, mode="linear", gated=False, extras=False)
    for k in ("u", "Bm", "Cm", "h0", "dy", "dhy"):
        c[k] = c[k].abs() + 0.25
    c["A"] = -torch.rand(20, N, generator=torch.Generator().manual_seed(seed)) - 0.1
    return c


def compare_infinite(c, dtype):
    """As compare, where the definition's values may be infinite or NaN: the same ones are."""
    got = ssm_run("linear", c)
    with np.errstate(all="ignore"):
        want = ssm_want("linear", c)
    for k, w in want.items():
        g, there = got[k].double().cpu().numpy(), np.isfinite(w.v)
        assert np.array_equal(g[~there], w.v[~there], equal_nan=True), (k, g[~there][:4], w.v[~there][:4])
        finite = torch.tensor(np.where(there, g, 0.0))
        check(k, finite, Bound(np.where(there, w.v, 0.0), np.where(there, w.e, 0.0)), "f32" if k in FP32 else dtype)
    return got, want


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_skip_that_is_left_out_takes_no_part(dtype):
    """Without D an infinite u or dy is no product with 0."""
    c = positive(72, 16, dtype, seed=12)
    c["u"][30, 1, 4] = float("inf")
    got, _ = compare_infinite(c, dtype)
    assert got["y"][30:, 1, 4].isinf().all() and not got["y"].isnan().any() and not got["hy"].isnan().any()
    g = {k: gpu(v) for k, v in c.items()}
    h, y = g["h0"].clone(), torch.empty_like(g["u"][0])
    R.rnn_ssm_step("linear", *(g[k] if k in ("A", "D", "delta_bias") or g[k] is None else g[k][30] for k in INPUTS), h, y, h)
    assert y[1, 4].isinf() and not y.isnan().any()
    c = positive(72, 16, dtype, seed=12)
    c["dy"][30, 1, 4] = float("inf")
    got = ssm_run("linear", c)
    assert got["du"][:31, 1, 4].isinf().all() and not got["du"].isnan().any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 13, 16, 24, 41, 64])
def test_infinite_inputs_are_infinite_results(dtype, N):
    """Also where the states are fewer than the lanes hold: those that are not there take no part."""
    c = positive(72, N, dtype, seed=12)
    c["u"][30, 1, 4] = float("inf")
    got, want = compare_infinite(c, dtype)
    for k in ("y", "hy", "ddelta", "dBm", "dCm", "dA"):
        assert got[k].isinf().any() and not got[k].isnan().any(), k
    assert got["y"][30:, 1, 4].isinf().all() and np.isinf(want["dA"].v[4]).all()
    c["delta"][40, 2, 7] = float("inf")
    got = ssm_run("linear", c)
    assert got["y"][40:, 2, 7].isinf().all() and got["hy"][2, 7].isinf().all()


@pytest.mark.parametrize("N", [1, 3, 13, 24])
def test_infinite_inputs_of_single_steps(N):
    c = positive(4, N, "f32", seed=13)
    c["u"][2, 1, 4], c["delta"][2, 2, 7] = float("inf"), float("inf")
    want = ssm_run("linear", c, backward=False)
    g = {k: gpu(v) for k, v in c.items()}
    h, y = g["h0"].clone(), torch.empty_like(g["u"])
    for t in range(4):
        R.rnn_ssm_step("linear", *(g[k] if k in ("A", "D", "delta_bias") or g[k] is None else g[k][t] for k in INPUTS), h, y[t], h)
    for b, e in ((1, 4), (2, 7)):
        assert y[2:, b, e].isinf().all() and h[b, e].isinf().all()
    assert torch.equal(y.isinf(), want["y"].isinf()) and not y.isnan().any() and int(y.isinf().sum()) == 4


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [1, 4, 13, 16, 64])
@pytest.mark.parametrize("T,lengths", [(70, None), (70, [70, 39, 1]), (300, [300, 203, 35])])
def test_infinite_states_past_a_rows_end(dtype, N, T, lengths):
    """A state that an infinite input has left infinite adds nothing past the row's last step, wherever that lies in a
    chunk of steps."""
    c = positive(T, N, dtype, seed=14)
    if lengths:
        c["lengths"] = torch.tensor(lengths, dtype=torch.int32)
    c["u"][30, 1, 4] = float("inf")
    got, want = compare_infinite(c, dtype)
    assert np.isinf(want["dA"].v[4]).all() and not got["dA"].isnan().any()
    c["u"][30, 1, 4], c["u"][-1 if not lengths else lengths[1] - 1, 1, 5] = 0.5, float("inf")     # the last step: dA is finite
    got, _ = compare_infinite(c, dtype)
    assert got["dA"].isfinite().all()


# (T, B, E, N, G): more channels a group than a workgroup takes, 256 with up to 4 states, 128 with 8, 64 with 16, 32 with 32
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,B,E,N,G,lengths", [(21, 2, 260, 4, 1, [21, 13]), (19, 1, 530, 3, 2, None), (33, 2, 130, 8, 1, [33, 6]),
                                               (40, 1, 300, 7, 1, None), (41, 2, 70, 16, 1, [41, 17]), (37, 2, 140, 16, 2, None),
                                               (50, 2, 200, 13, 1, [0, 50]), (26, 2, 33, 30, 1, [26, 9]), (35, 1, 140, 32, 2, None),
                                               (30, 2, 40, 64, 1, [30, 23])])
def test_sums_over_several_workgroups(dtype, T, B, E, N, G, lengths):
    """dB and dC of a group that several workgroups share, for every number of lanes a channel."""
    print("CASE ssm sums", dtype, T, B, E, N, G, flush=True)
    compare("softplus", ssm_case(T, B, E, N, G, dtype, lengths, seed=15), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,B,E,N,G,lengths", [(520, 2, 90, 16, 1, [520, 301]), (300, 1, 300, 4, 1, None), (200, 1, 150, 8, 1, [130])])
def test_sums_over_several_workgroups_and_segments(dtype, T, B, E, N, G, lengths):
    compare("softplus", ssm_case(T, B, E, N, G, dtype, lengths, seed=16), dtype)


@pytest.mark.parametrize("dtype,E,N,G", [("f32", 11040, 16, 10), ("bf16", 44160, 3, 1)])
def test_sums_over_several_workgroups_and_parts(dtype, E, N, G):
    """690 waves a segment: backward has two segments, cut into two parts each for its first launch, as in wide training
    batches, and several workgroups a group."""
    print("CASE ssm parts", dtype, E, N, G, flush=True)
    compare("softplus", ssm_case(130, 1, E, N, G, dtype, [117], seed=17), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [4, 13, 16])
def test_infinite_states_stay_infinite_over_segments(dtype, N):
    """Segments whose decay is far below fp32's range, after an infinite input or before an infinite gradient: infinity
    times a decay, not times 0."""
    c = positive(400, N, dtype, seed=18)
    c["A"] *= 20.0
    c["delta"][:] = 0.5
    c["u"][30, 1, 4] = float("inf")
    got, _ = compare_infinite(c, dtype)
    assert got["y"][30:, 1, 4].isinf().all() and got["hy"][1, 4].isinf().all()
    c["u"][30, 1, 4], c["dhy"][1, 5] = 0.5, float("inf")
    got = ssm_run("linear", c)
    assert got["dh0"][1, 5].isinf().all() and got["du"][:, 1, 5].isinf().all()
