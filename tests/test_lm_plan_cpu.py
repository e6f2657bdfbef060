"""The feed-forward products' planner, on the host."""

import pytest

from tests import lm_plan


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    return lm_plan.build(tmp_path_factory.mktemp("plan"))


def test_places_fit_the_lds(probe):
    """As many workgroups as the model takes a CU to hold fit its LDS."""
    got = lm_plan.rows(probe, "places")
    assert len(got) == 6
    for glu, tile, places, lds, cu in got:
        assert places >= 1 and places * lds <= cu == 160 * 1024, (glu, tile)
