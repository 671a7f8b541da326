"""pa_pool_check where a step ran out of blocks and another call saw what does not fit: each is told, one call after the other."""
import pytest
import torch

from paged_kv_cache_223_gb300 import pagedattn as pa
from test_gpu_step_tables import State

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("order", ["blocks first", "bounds first"])
def test_out_of_blocks_is_told_beside_bounds(order):
    s = State([16, 15], 8, 4, 16)
    steps = [([1, 18], pa.PA_ERR_OOM), ([-1, 0], pa.PA_ERR_DEVICE_BOUNDS)]
    for new, _ in steps if order == "blocks first" else steps[::-1]:
        s.call(new, 19)
    assert [s.pool.check() for _ in range(4)] == [pa.PA_ERR_DEVICE_BOUNDS, pa.PA_ERR_OOM, pa.PA_OK, pa.PA_OK]
    s.check((), ())
    for new, status in steps:                              # alone
        s.call(new, 19)
        assert s.pool.check() == status and s.pool.check() == pa.PA_OK


def test_a_timeout_beside_both():
    s = State([16, 15], 8, 4, 16)
    s.call([1, 18], 19), s.call([-1, 0], 19)
    assert pa.lib().pa_pool_selftest_wait(s.pool.handle, 1000, None) == pa.PA_OK
    torch.cuda.synchronize()
    assert [s.pool.check() for _ in range(3)] == [pa.PA_ERR_TIMEOUT, pa.PA_ERR_OOM, pa.PA_OK]


def test_its_words():
    assert "blocks" in pa.status_string(pa.PA_ERR_OOM)
