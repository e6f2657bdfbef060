"""The feed-forward products' planner, on the host."""

import pytest

from tests import lm_plan, lm_tile_cases


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    return lm_plan.build(tmp_path_factory.mktemp("plan"))


def test_places_fit_the_lds(probe):
    """As many workgroups as the model takes a CU to hold fit its LDS."""
    got = lm_plan.rows(probe, "places")
    assert len(got) == 6
    for glu, tile, places, lds, cu in got:
        assert places >= 1 and places * lds <= cu == 160 * 1024, (glu, tile)


def test_the_listed_sizes_run_every_tile(probe):
    """All that the planner can choose: for each type and product, each tile with k whole, and each that may be split
    with k split."""
    ran = set()
    sizes = lm_tile_cases.SIZES
    for (_, _, _, bf), (g, gs, d, y, ys, q, *qs) in zip(sizes, lm_plan.rows(probe, *[v for s in sizes for v in s])):
        ran |= {("gated", bf, g, gs > 1), ("dgated", bf, d, False), ("y", bf, y, ys > 1)}
        ran |= {(k, bf, q, n > 1) for k, n in zip(("dx", "dw_in", "dw_out"), qs)}
    want = {(k, bf, t, False) for k in ("gated", "dgated", "y", "dx", "dw_in", "dw_out") for bf, tiles in
            ((0, (128, 64)), (1, (256, 128, 64))) for t in tiles}
    want |= {(k, bf, t, True) for k in ("gated", "y", "dx", "dw_in", "dw_out") for bf in (0, 1) for t in (128, 64)}
    assert ran == want, (want - ran, ran - want)
