"""Causal convolution on the GPU against the definition in 64 bits; tolerances are the oracle's bounds on an evaluation in
fp32 and half a step of the output's type."""

import pytest
import torch

import layer_rnn_forward_amd as R
from oracle.bounds import check
from tests.block_gpu import conv_case, conv_run, conv_want, room

pytestmark = pytest.mark.gpu
FP32 = ("dw", "dbias")


def compare(act, c, dtype, wide=0):
    got, want = conv_run(act, c, wide), conv_want(act, c)
    for k, v in want.items():
        check(k, got[k], v, "f32" if k in FP32 else dtype)
    return got


@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,B,C,K", [(1, 1, 1, 4), (2, 3, 5, 4), (7, 2, 64, 3), (33, 2, 260, 4), (8, 1, 256, 2), (65, 3, 17, 8), (40, 2, 30, 1),
                                     (130, 1, 258, 5), (31, 2, 9, 6), (70, 2, 12, 7)])
def test_sequences(act, dtype, T, B, C, K):
    print("CASE conv", act, dtype, T, B, C, K, flush=True)
    compare(act, conv_case(T, B, C, K, dtype), dtype)


@pytest.mark.parametrize("dtype,K,act", [("f32", 3, "none"), ("bf16", 2, "silu")])
def test_long_pieces(dtype, K, act):
    """So many rows that a wave walks pieces of more than 8 steps; rows that end inside, at and before their ends."""
    lengths = [300, 0, 1, 16, 17, 8, 24, 299] + [300 - i for i in range(84)]
    compare(act, conv_case(300, 92, 257, K, dtype, lengths), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,K,lengths", [(40, 4, [40, 0, 1, 2, 3, 17]), (9, 8, [9, 8, 7, 1, 0, 3]), (70, 3, [-5, 99, 64, 32, 33, 31])])
def test_ragged_rows(dtype, T, K, lengths):
    """Lengths within, below and above the range; what lies past a row's length is not used."""
    c = conv_case(T, 6, 70, K, dtype, lengths)
    got = compare("silu", c, dtype)
    for b, n in enumerate(lengths):
        for k in ("x", "dy"):
            c[k][max(n, 0):, b] = float("nan")
    again = conv_run("silu", c)
    for k in got:
        assert torch.equal(got[k], again[k]), k


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B", [1, 3])
def test_slices_of_wider_tensors(dtype, B):
    for T in (1, 35):
        c = conv_case(T, B, 66, 4, dtype)
        got, want = compare("silu", c, dtype, wide=9), conv_run("silu", c)
        for k in want:
            assert torch.equal(got[k], want[k]), k


def test_without_bias_and_state():
    for act in ("silu", "none"):
        compare(act, conv_case(50, 2, 40, 4, "f32", bias=False, state=False), "f32")


def test_no_steps():
    c = conv_case(0, 2, 10, 4, "f32")
    got = compare("silu", c, "f32")
    assert torch.equal(got["sy"].cpu(), c["s0"]) and torch.equal(got["ds0"].cpu(), c["dsy"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1, 2, 4, 7])
def test_steps_follow_the_sequence(dtype, K):
    """Single steps, the state updated in place, and a sequence in two pieces: bitwise the sequence's results."""
    c = conv_case(45, 3, 77, K, dtype)
    want = conv_run("silu", c)
    g = {k: v.cuda() if v is not None else None for k, v in c.items()}
    s, y = g["s0"].clone(), torch.empty_like(g["x"])
    for t in range(45):
        R.rnn_conv_step("silu", g["x"][t], g["w"], g["bias"], s, y[t], s)
    assert torch.equal(y, want["y"]) and torch.equal(s, want["sy"])
    s = g["s0"].clone()
    for a, b in ((0, 2), (2, 45)):
        R.rnn_conv_forward("silu", g["x"][a:b], g["w"], g["bias"], s, None, y[a:b], s)
    assert torch.equal(y, want["y"]) and torch.equal(s, want["sy"])


def test_step_on_slices():
    c = conv_case(1, 5, 40, 4, "bf16")
    g = {k: v.cuda() if v is not None else None for k, v in c.items()}
    wide, out = torch.randn(5, 90, device="cuda").bfloat16(), torch.zeros(5, 60, device="cuda", dtype=torch.bfloat16)
    wide[:, 3:43] = g["x"][0]
    y, sy = torch.empty(5, 40, device="cuda", dtype=torch.bfloat16), torch.empty_like(g["s0"])
    R.rnn_conv_step("none", g["x"][0], g["w"], None, None, y, None)
    R.rnn_conv_step("none", wide[:, 3:43], g["w"], None, None, out[:, 20:], sy)
    assert torch.equal(out[:, 20:], y) and not out[:, :20].any() and torch.equal(sy[-1], g["x"][0]) and not sy[:-1].any()


def test_not_wanted_gradients():
    c = conv_case(60, 2, 90, 4, "bf16")
    want = conv_run("silu", c)
    g = {k: v.cuda() if v is not None else None for k, v in c.items()}
    names = ("dx", "dw", "dbias", "ds0")
    for name in names:
        out = [torch.empty_like(want[k]) if k == name else None for k in names]
        R.rnn_conv_backward("silu", g["x"], g["w"], g["bias"], g["s0"], None, g["dy"], g["dsy"], *out, room(R.rnn_conv_workspace_size(60, 2, 90, 4)))
        assert torch.equal(out[names.index(name)], want[name]), name


def test_no_rows():
    """The parameters' gradients over no rows are zero."""
    x, w = torch.empty(4, 0, 6, device="cuda"), torch.ones(6, 3, device="cuda")
    dw, db = torch.full_like(w, 3.0), torch.full((6,), 3.0, device="cuda")
    R.rnn_conv_backward("silu", x, w, None, None, None, x, None, None, dw, db, None, room(R.rnn_conv_workspace_size(4, 0, 6, 3)))
    assert not dw.any() and not db.any()


def test_more_channels_than_32_bits_of_weights():
    """C * K past 2^31: a step without state or bias is the product with the newest input's weight, exactly."""
    C, K = (1 << 28) + 5, 8
    x, w = torch.empty(1, 1, C, device="cuda").uniform_(-1, 1), torch.empty(C, K, device="cuda").uniform_(-1, 1)
    y = torch.full_like(x, 7.0)
    R.rnn_conv_forward("none", x, w, None, None, None, y, None)
    assert torch.equal(y.view(C), w[:, K - 1] * x.view(C))


def test_more_threads_of_sums_than_a_dimension_takes():
    """(K + 1) C past 2^28: the sums of dw and dbias have more than 2^32 threads."""
    T, C, K = 2, 1 << 26, 4
    x, dy = (torch.empty(T, 1, C, device="cuda").uniform_(-1, 1) for _ in range(2))
    w, dw, db = torch.ones(C, K, device="cuda"), torch.full((C, K), 7.0, device="cuda"), torch.full((C,), 7.0, device="cuda")
    R.rnn_conv_backward("none", x, w, None, None, None, dy, None, None, dw, db, None, room(R.rnn_conv_workspace_size(T, 1, C, K)))
    x, dy = x.view(T, C), dy.view(T, C)
    assert torch.equal(db, dy[0] + dy[1]) and not dw[:, :2].any() and torch.equal(dw[:, 2], dy[1] * x[0])
    a, b = dy[0].double() * x[0], dy[1].double() * x[1]
    # one product rounded, then their sum: half a step (2^-24) of each
    assert ((dw[:, 3] - (a + b)).abs() <= 2.0 ** -24 * (2 * a.abs() + b.abs()) * (1 + 2.0 ** -20)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", [40, 256])
def test_steps_past_a_row_take_no_part_in_gradients(dtype, C):
    """An infinite last input of a row meets the newest tap only; an infinite weight leaves dx past the row's length 0."""
    c = conv_case(45, 3, C, 4, dtype, [45, 21, 1], bias=False)
    c["dy"] = c["dy"].abs() + 0.1
    c["x"][20, 1] = c["s0"][1, 2] = 0
    want = conv_run("none", c)
    c["x"][20, 1] = c["s0"][1, 2] = float("inf")      # the second row's last; the third's x_-2, which its one step meets with tap 1
    got = conv_run("none", c)
    assert torch.equal(got["dw"][:, [0, 2]], want["dw"][:, [0, 2]])
    assert (got["dw"][:, [1, 3]] == float("inf")).all()
    for k in ("dx", "ds0", "dbias"):
        assert torch.equal(got[k], want[k]), k
    c["w"][:, 2] = float("inf")
    got = conv_run("none", c)
    for b, n in enumerate((45, 21, 1)):
        assert not got["dx"][n:, b].any() and not got["y"][n:, b].any()


@pytest.mark.parametrize("dtype,K,act", [("f32", 6, "silu"), ("bf16", 7, "none"), ("f32", 8, "silu"), ("bf16", 8, "silu")])
def test_long_pieces_of_wide_filters(dtype, K, act):
    """Whole groups of steps without branches, whose first ones wait for K - 1 steps, for the widest filters."""
    lengths = [300, 0, 1, 16, 17, 8, 24, 299] + [300 - i for i in range(84)]
    compare(act, conv_case(300, 92, 257, K, dtype, lengths, seed=2), dtype)
