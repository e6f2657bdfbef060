"""The feed-forward block on every tile of every product, with k whole and split (odd widths, ragged last tiles), against
its float64 definition; tolerances as in the block's own tests."""

import pytest

from tests import lm_tile_cases
from tests import test_gpu_lm_ffn as ffn

pytestmark = pytest.mark.gpu


@pytest.mark.timeout(300)
@pytest.mark.parametrize("act,save", [("silu", "none"), ("silu", "full"), ("gelu", "int8")])
@pytest.mark.parametrize("size", lm_tile_cases.SIZES, ids=lambda s: "x".join(map(str, s)))
def test_tiles(size, act, save):
    print("CASE ffn tiles", size, act, save, flush=True)
    c = ffn.make(*size[:3], "bf16" if size[3] else "f32")
    ffn.check(ffn.run(c, act, save), ffn.expected(c, act, save), c)
