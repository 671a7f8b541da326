"""select_blocks of contexts that the budget holds whole: every block is listed, and an id outside the pool is flagged there too."""
import numpy as np
import pytest

from paged_kv_cache_223_gb300 import pagedattn as pa
from test_gpu_select_blocks import buffer, expected, i32, make, torch

pytestmark = pytest.mark.gpu


# one CTA to a sequence, and (one sequence of long rows) a cluster
@pytest.mark.parametrize("lens,stride", [([900, 300, 16, 0], 60), ([5000], 20000)])
@pytest.mark.parametrize("bad", [-1, 10 ** 6, 2 ** 31 - 1])
def test_ids_outside_the_pool_are_flagged(lens, stride, bad):
    pool, codes, steps, tables, q = make(lens, 8, 2, 64, torch.float16, 16, seed=1, stride=stride)
    want = expected(q, codes, steps, tables, lens, 16, 400, 1, 2)
    got = pool.select_blocks(q, buffer(codes, steps), tables, i32(lens), 400)      # -1 behind the context: nothing is flagged
    assert pool.check() == pa.PA_OK and np.array_equal(got.cpu().numpy(), want)
    for at in (0, -(-lens[0] // 16) - 1):
        wrong = tables.clone()
        wrong[0, at] = bad
        got = pool.select_blocks(q, buffer(codes, steps), wrong, i32(lens), 400)
        assert pool.check() == pa.PA_ERR_DEVICE_BOUNDS
        assert np.array_equal(got.cpu().numpy(), want)
