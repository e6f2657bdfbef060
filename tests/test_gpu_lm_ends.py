"""Infinities in the feed-forward block where F is no whole number of 16-byte pieces: what lies past a row's last column
inside the library's own buffers must not turn them into NaN."""

import pytest
import torch

import layer_rnn_forward_amd as R
from tests import test_gpu_lm_ffn as ffn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,F", [(3, 33), (100, 33), (100, 70), (300, 129), (100, 64), (70, 2501)])
@pytest.mark.parametrize("save", ["none", "full", "int8"])
def test_an_infinite_row_is_infinite(dtype, M, F, save):
    """All values positive: an infinity in a row of x makes that row of y infinite, one in dy that row of dx; the other
    rows keep theirs."""
    D = 40
    print("CASE ffn ends", dtype, M, F, save, flush=True)
    t = ffn.DT[dtype]
    gen = torch.Generator(device="cuda").manual_seed(1)

    def positive(*shape):
        return (torch.rand(shape, device="cuda", generator=gen) + 0.25).to(t)

    x, w_in, w_out, dy = positive(M, D), positive(2 * F, D), positive(D, F), positive(M, D)
    ws = torch.empty(R.rnn_ffn_workspace_size(M, D, F, dtype, save), dtype=torch.uint8, device="cuda")
    reserve = torch.empty(R.rnn_ffn_reserve_size(M, D, F, dtype, save), dtype=torch.uint8, device="cuda")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    others = torch.arange(M, device="cuda") != 1
    bad = x.clone()
    bad[1, 3] = float("inf")
    R.rnn_ffn_forward("silu", bad, w_in, w_out, y, ws, save, reserve)
    assert (y[1] == float("inf")).all() and torch.isfinite(y[others]).all()
    if save == "none":
        return
    R.rnn_ffn_forward("silu", x, w_in, w_out, y, ws, save, reserve)
    assert torch.isfinite(y).all()
    dy[1, 3] = float("inf")
    R.rnn_ffn_backward("silu", x, w_in, w_out, dy, dx, None, None, ws, save, reserve)
    assert (dx[1] == float("inf")).all() and torch.isfinite(dx[others]).all()
