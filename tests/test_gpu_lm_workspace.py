"""One workspace and reserve, sized for the largest batch, for every smaller one: bitwise the results of its own."""

import pytest
import torch

import layer_rnn_forward_amd as R
from tests import test_gpu_lm_ffn as ffn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,save", [("f32", "none"), ("bf16", "none"), ("f32", "full"), ("bf16", "int8")])
@pytest.mark.parametrize("D,F", [(512, 1024), (77, 2050)])
def test_a_workspace_for_the_largest_batch(dtype, save, D, F):
    most = 400
    ws = torch.full((R.rnn_ffn_workspace_size(most, D, F, dtype, save),), 0x7F, dtype=torch.uint8, device="cuda")
    reserve = torch.full((R.rnn_ffn_reserve_size(most, D, F, dtype, save),), 0x7F, dtype=torch.uint8, device="cuda")
    for M in (1, 64, 65, 129, 200, 400):
        print("CASE ffn workspace", dtype, save, D, F, M, flush=True)
        c = ffn.make(M, D, F, dtype)
        want = ffn.run(c, "silu", save)
        x, w_in, w_out, dy = (ffn.dev(c, k) for k in ("x", "w_in", "w_out", "dy"))
        got = {k: torch.zeros_like(v) for k, v in want.items()}
        R.rnn_ffn_forward("silu", x, w_in, w_out, got["y"], ws, save, reserve)
        if save != "none":
            R.rnn_ffn_backward("silu", x, w_in, w_out, dy, got["dx"], got["dw_in"], got["dw_out"], ws, save, reserve)
        for k, v in want.items():
            assert torch.equal(got[k], v), (M, k)
