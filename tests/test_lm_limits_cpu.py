"""Sizes at the ends of the language-model operators' ranges: refused, or with a workspace of the size that the
layout gives, without a GPU."""

import ctypes

import pytest

import layer_rnn_forward_amd as R

UNSUPPORTED = -2


@pytest.mark.parametrize("T,want", [(0x7fffffff, UNSUPPORTED), (0x7fffffff - 1023, UNSUPPORTED), (0x7fffffff - 1024, 0)])
def test_longest_sequences(T, want):
    n = ctypes.c_size_t()
    assert R.load_library().rnn_scan_workspace_size(T, 1, 1, 1, ctypes.byref(n)) == want


def test_workspaces_of_large_problems_do_not_wrap():
    # a state before every 8th step: 4 bytes for 8 values
    assert R.rnn_scan_workspace_size(1 << 30, 4, 1 << 20, 2) >= (1 << 30) * (1 << 23) // 2
    # the projections in 16 bits each and the gated product in bf16
    assert R.rnn_ffn_reserve_size(1 << 29, 1 << 10, 1 << 19, "bf16", "full") >= 6 * (1 << 48)
    assert R.rnn_checkpoint_size(0x7fffffff, 1 << 29) > (1 << 59)


def test_sizes_beyond_a_c_int_are_refused():
    for call in (lambda: R.rnn_scan_workspace_size(1, 1 << 32, 1), lambda: R.rnn_ffn_workspace_size(1 << 31, 8, 8, "bf16"),
                 lambda: R.rnn_ffn_reserve_size(1, 1 << 33, 8, "f32", "full"), lambda: R.rnn_checkpoint_size(1 << 32, 4),
                 lambda: R.rnn_checkpoint_size(4, -(1 << 32))):
        with pytest.raises(ValueError, match="C int"):
            call()
    with pytest.raises(R.RNNError):
        R.rnn_checkpoint_size(-1, 4)
