"""Sizes of the state-space block's workspaces: one that is sized for the longest sequences and the largest batch does for
all others, without a GPU."""

import random

import pytest

import layer_rnn_forward_amd as R


def falls(size, steps):
    last, at = -1, None
    for n in steps:
        s = size(n)
        if s < last:
            return f"{n}: {s}, {at}: {last}"
        last, at = s, n
    return None


STEPS = [*range(0, 1500), *range(1500, 9000, 7), *range(9000, 300000, 4099)]
ROWS = [*range(0, 300), *range(300, 5000, 37)]


@pytest.mark.parametrize("save", ["none", "full"])
@pytest.mark.parametrize("E,N,G", [(1760, 16, 1), (64, 16, 1), (357, 13, 3), (2048, 16, 1), (16, 4, 1), (3520, 1, 1), (40, 64, 4),
                                   (20000, 16, 1), (4096, 32, 1)])
def test_ssm_sizes_grow_with_steps_and_rows(E, N, G, save):
    for B in (1, 2, 3, 7, 32):
        assert falls(lambda T: R.rnn_ssm_workspace_size(T, B, E, N, G, save), STEPS) is None, B
    for T in (0, 1, 31, 64, 100, 613, 2048, 16384):
        assert falls(lambda B: R.rnn_ssm_workspace_size(T, B, E, N, G, save), ROWS) is None, T


@pytest.mark.parametrize("C,K", [(1760, 4), (64, 4), (357, 3), (2048, 4), (16, 8), (3520, 2), (20000, 1)])
def test_conv_sizes_grow_with_steps_and_rows(C, K):
    for B in (1, 2, 3, 7, 32):
        assert falls(lambda T: R.rnn_conv_workspace_size(T, B, C, K), STEPS) is None, B
    for T in (0, 1, 8, 31, 64, 100, 613, 2048, 16384):
        assert falls(lambda B: R.rnn_conv_workspace_size(T, B, C, K), ROWS) is None, T


def test_norm_sizes_grow_with_rows():
    for D in (1, 64, 1357, 2048, 8195, 16384, 40000):
        assert falls(lambda M: R.rnn_norm_workspace_size(M, D), STEPS) is None, D


def test_sizes_grow_at_random():
    rng = random.Random(5)
    for _ in range(200):
        G, N = rng.choice([1, 1, 2, 4]), rng.randint(1, 64)
        E, K, save = G * int(2 ** rng.uniform(0, 12)), rng.randint(1, 8), rng.choice(["none", "full"])
        pairs = [(0, 0)]
        for _ in range(30):
            pairs.append((pairs[-1][0] + int(2 ** rng.uniform(0, 10)) - 1, pairs[-1][1] + int(2 ** rng.uniform(0, 3)) - 1))
        assert falls(lambda p: R.rnn_ssm_workspace_size(*p, E, N, G, save), pairs) is None, (E, N, G, save)
        assert falls(lambda p: R.rnn_conv_workspace_size(*p, E, K), pairs) is None, (E, K)


def test_no_more_is_reserved_than_the_passes_hold():
    """A training batch: the states before every 8th step, the sums of dB and dC over 64 channels at a time, and little
    more; inference keeps maps of segments alone, and many rows none but their own."""
    T, B, E, N = 2048, 8, 2048, 16
    own = T // 8 * B * E * N * 4 + T * B * 2 * N * (E // 64) * 4
    assert own <= R.rnn_ssm_workspace_size(T, B, E, N, 1, "full") <= own + (16 << 20)
    assert R.rnn_ssm_workspace_size(T, B, E, N) <= 8 << 20
    assert R.rnn_ssm_workspace_size(T, 1000, E, N) <= 8 << 20
    assert R.rnn_ssm_workspace_size(1, 16, E, N) <= 256
    assert R.rnn_conv_workspace_size(T, B, E, 4) <= 8 << 20
