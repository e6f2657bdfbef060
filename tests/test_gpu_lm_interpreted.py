"""The operators through the interpreted path (no compiled entries): bitwise the results of the compiled one."""

import pytest
import torch

from layer_rnn_forward_amd import _binding
from tests import test_gpu_lm_checkpoint as ckpt
from tests import test_gpu_lm_ffn as ffn
from tests import test_gpu_lm_scan as scan

pytestmark = pytest.mark.gpu


def passes():
    c = scan.make("gated", "bf16", 300, 2, 64, 2, [300, 17])
    out = {f"scan.{k}": v for k, v in scan.run(c).items()}
    hy = torch.empty(3, 16, device="cuda")
    _binding.rnn_scan_step("linear", torch.arange(96, device="cuda").view(3, 32).float(), None, None, hy)
    out["step"] = hy
    f = ffn.make(100, 64, 96, "bf16")
    for save in ("none", "full", "int8"):
        out |= {f"ffn.{save}.{k}": v for k, v in ffn.run(f, "silu", save).items()}
    out["checkpoint"] = ckpt.there_and_back(torch.arange(2000, device="cuda").view(40, 50).float())
    return out


def test_interpreted_calls(monkeypatch):
    want = passes()
    assert type(_binding._CALL).__name__ == "module", "the compiled entries are not built"
    monkeypatch.setattr(_binding, "_CALL", _binding._Interpreted("a test"))
    with pytest.warns(RuntimeWarning, match="_call.so"):
        got = passes()
    assert got.keys() == want.keys()
    for k, v in want.items():
        assert torch.equal(got[k], v), k
