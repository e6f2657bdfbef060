"""rnn_scan_status without a GPU: what it refuses before anything is read."""

import ctypes

import pytest
import torch

import layer_rnn_forward_amd as R

SOME = 1 << 20


def test_refusals():
    lib = R.load_library()
    for args in ((None, None, 512), (None, SOME + 4, 512), (None, SOME, 255)):
        assert lib.rnn_scan_status(*args[:2], ctypes.c_size_t(args[2])) == -1, args
    with pytest.raises(ValueError, match="device"):
        R.rnn_scan_status(torch.zeros(512, dtype=torch.uint8))
    with pytest.raises(TypeError):
        R.rnn_scan_status(None)
