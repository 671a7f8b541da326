"""key_bounds of blocks that were filled without it: a call that counts their tokens among the newest makes their bounds anew."""
import numpy as np
import pytest
import torch

from paged_kv_cache_223_gb300 import pagedattn as pa
from test_gpu_key_bounds import expected, i32, make, parts, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,d,fp8", [(torch.bfloat16, 64, False), (torch.float16, 128, True)])
def test_a_copied_block(dt, d, fp8):
    pool, rows, bounds = make([90, 40], 2, d, dt, 16, fp8)
    run(pool, rows, bounds, [90, 40], [90, 40])
    src, dst = rows[0][2], rows[1][1]
    pa.copy_blocks(pool, i32([[src, dst]]))
    was = [x.cpu().numpy().copy() for x in parts(pool, bounds)]
    pool.key_bounds(bounds, i32([0, 1, 2]), i32(rows), i32([90, 40]), 2)       # the newest tokens: not that block
    now = [x.cpu().numpy() for x in parts(pool, bounds)]
    assert np.array_equal(now[0], was[0]) and np.array_equal(now[1], was[1]) and not np.array_equal(was[0][src], was[0][dst])
    want = run(pool, rows, bounds, [0, 40], [90, 40])                           # its tokens among the newest
    assert np.array_equal(want[0][src], want[0][dst]) and np.array_equal(want[1][src], want[1][dst])
    whole = expected(pool, bounds, [0, 90, 130], rows, [90, 40])                # every block of both contexts: nothing changes
    assert np.array_equal(whole[0], want[0]) and np.array_equal(whole[1], want[1])
    assert pool.check() == pa.PA_OK
