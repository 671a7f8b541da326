"""More host-side refusals of the serving operators, and their limits as the header states them."""

import pytest

from paged_kv_cache_223_gb300 import _build


@pytest.fixture(scope="module")
def pa():
    _build.build_cuda()
    from paged_kv_cache_223_gb300 import pagedattn
    return pagedattn


@pytest.mark.parametrize("rot", [1, 17, 33, 127])
def test_a_base_gives_frequencies_of_whole_pairs(pa, rot):
    with pytest.raises(ValueError):
        pa.Rope.from_base(rot)
