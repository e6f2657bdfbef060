"""8-bit checkpoints on the GPU: every value has to be the definition's (whole numbers of a power of two)."""

import numpy as np
import pytest
import torch

import layer_rnn_forward_amd as R
from oracle import lm_oracle as O

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def there_and_back(x, out_dtype=None):
    kept = torch.full((R.rnn_checkpoint_size(*x.shape) + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    R.rnn_checkpoint_store(x, kept)
    assert (kept[-64:] == 0x5A).all()                  # nothing is written past the queried size
    back = torch.full(x.shape, 9.0, dtype=out_dtype or x.dtype, device="cuda")
    R.rnn_checkpoint_load(kept, back)
    return back


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 31), (2, 32), (5, 33), (7, 64), (20, 800), (9, 357), (1, 5000),
                                       (4099, 8), (1000, 1), (130, 1024), (65, 40), (33, 16), (64, 2048)])
def test_values(dtype, rows, cols):
    print("CASE checkpoint", dtype, rows, cols, flush=True)
    rng = np.random.default_rng([rows, cols])
    x = rng.normal(size=(rows, cols)) * np.exp2(rng.normal(size=(rows, 1)) * 20)
    x[rng.random(size=x.shape) < 0.1] = 0
    x = torch.tensor(x).to(DT[dtype])
    want = O.checkpoint_round(x.double().numpy())
    for out in DT.values():
        assert np.array_equal(there_and_back(x.cuda(), out).double().cpu().numpy(), want)


def test_ties_borders_and_small_values():
    rows = [[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, 126.5, -126.5],       # ties to even
            [127.5, 127.75, -127.9, 1.0, 0.0, -0.0, 64.0, 63.5],     # saturation just under the next power
            [128.0, 1.0, 3.0, -1.0, -3.0, 5.0, 127.0, 2.0],
            [2.0 ** -126, 2.0 ** -127, 2.0 ** -149, 0, 0, 0, 0, 0],  # subnormal values and units
            [2.0 ** -120, 2.0 ** -126, 2.0 ** -127, 3 * 2.0 ** -127, 0, 0, 0, 0],
            [3.0e38, -3.3e38, 1.0e37, 0, 0, 0, 0, 1.0]]
    x = torch.tensor(rows, dtype=torch.float64).float()
    got = there_and_back(x.cuda()).double().cpu().numpy()
    assert np.array_equal(got, O.checkpoint_round(x.double().numpy()))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_infinities_and_nans_mark_their_group(dtype):
    x = torch.randn(40, 100).to(DT[dtype])
    x[3, 40], x[7, 99], x[9, 0] = float("inf"), float("nan"), -float("inf")
    got = there_and_back(x.cuda()).double().cpu().numpy()
    assert np.array_equal(got, O.checkpoint_round(x.double().numpy()), equal_nan=True)
    assert np.isnan(got).sum() == 32 + 4 + 32


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [64, 77])
def test_misaligned_tensors(dtype, cols):
    x = torch.randn(50, cols, device="cuda").to(DT[dtype])
    want = there_and_back(x)
    buf = torch.empty(50 * cols + 1, dtype=x.dtype, device="cuda")
    buf[1:] = x.reshape(-1)
    kept = torch.empty(R.rnn_checkpoint_size(50, cols), dtype=torch.uint8, device="cuda")
    R.rnn_checkpoint_store(buf[1:].view(50, cols), kept)
    back = torch.zeros_like(buf)
    R.rnn_checkpoint_load(kept, back[1:].view(50, cols))
    assert torch.equal(back[1:].view(50, cols), want) and back[0] == 0


def test_empty():
    for shape in ((0, 5), (5, 0), (0, 0)):
        assert there_and_back(torch.empty(shape, device="cuda")).shape == shape


def test_graph_and_stream():
    x = torch.randn(300, 500, device="cuda")
    want = there_and_back(x)
    kept = torch.empty(R.rnn_checkpoint_size(300, 500), dtype=torch.uint8, device="cuda")
    back = torch.zeros_like(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        R.rnn_checkpoint_store(x, kept)
        R.rnn_checkpoint_load(kept, back)
    for _ in range(3):
        back.zero_()
        kept.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(back, want)


@pytest.mark.timeout(300)
def test_offsets_past_32_bits():
    rows, cols = 270000, 8000
    print("CASE checkpoint past 32 bits", flush=True)
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda").normal_()
    assert x.numel() > 1 << 31
    back = there_and_back(x)
    for r in (0, 131071, rows - 3):
        want = O.checkpoint_round(x[r:r + 3].double().cpu().numpy())
        assert np.array_equal(back[r:r + 3].double().cpu().numpy(), want)
