"""Sizes of the operators' workspaces: what a server that sizes once for its largest batch relies on, without a GPU."""

import random

import pytest

import layer_rnn_forward_amd as R


def sizes(rng):
    es = rng.choice(["f32", "bf16"])
    D, F = (int(2 ** rng.uniform(3, 13)) for _ in range(2))
    return D, F, es, rng.choice(["none", "full", "int8"])


def falls(D, F, es, save, rows):
    last, at = -1, 0
    for M in rows:
        n = R.rnn_ffn_workspace_size(M, D, F, es, save)
        if n < last:
            return f"{M} rows {n}, {at} rows {last}"
        last, at = n, M
    return None


@pytest.mark.parametrize("D,F,es,save", [(4096, 4096, "f32", "none"), (2048, 8192, "bf16", "none"), (128, 256, "bf16", "full"),
                                         (357, 1021, "f32", "full"), (1760, 7040, "bf16", "int8"), (33, 5001, "f32", "int8"),
                                         (2040, 130, "f32", "none"), (8, 8, "bf16", "full"), (1, 4096, "bf16", "none")])
def test_more_rows_never_need_less(D, F, es, save):
    rows = [*range(0, 2300), *range(2300, 40000, 61), *range(40000, 200000, 4099)]
    assert falls(D, F, es, save, rows) is None


def test_more_rows_never_need_less_at_random_sizes():
    rng = random.Random(3)
    for _ in range(120):
        c = sizes(rng)
        rows = sorted({0, 64, 65, *(int(2 ** rng.uniform(0, 17)) for _ in range(60))})
        assert falls(*c, rows) is None, c


def test_few_rows_do_not_reserve_the_weights():
    assert R.rnn_ffn_workspace_size(1, 2048, 8192, "bf16") == 2 * 8192 * 2
    assert R.rnn_ffn_workspace_size(64, 2048, 8192, "bf16") == 64 * 2 * 8192 * 2
    assert R.rnn_ffn_workspace_size(0, 2048, 8192, "bf16") == 256


def test_large_calls_reserve_little_more_than_they_use():
    """Beyond the buffers that a call of these sizes may write: 64 MiB of partial sums at most."""
    for M, D, F, save in ((8192, 2048, 8192, "full"), (6000, 1760, 7040, "int8"), (6000, 800, 3200, "none")):
        own = 2 * (M * D + 2 * F * D + D * F)
        own += 2 * M * F if save != "full" else 0
        own += 2 * (M * D + 2 * M * F) if save != "none" else 0
        assert own <= R.rnn_ffn_workspace_size(M, D, F, "bf16", save) <= own + (64 << 20) + 4096


def test_scan_workspaces_grow():
    rng = random.Random(4)
    for _ in range(60):
        B, H, d = rng.randint(1, 9), rng.randint(1, 300), rng.choice([1, 2])
        n = [R.rnn_scan_workspace_size(T, B, H, d) for T in range(0, 3000, 7)]
        assert n == sorted(n)
