"""step_tables: a step that would put an id outside the pool back on the free stack is refused, so that no other sequence takes it."""
import pytest
import torch

from paged_kv_cache_223_gb300 import pagedattn as pa
from test_gpu_step_tables import State

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 6000, 2 ** 31 - 1])
@pytest.mark.parametrize("b,at,spare", [(0, 2, 0), (150, 5, 3), (299, 1, 40000)])
def test_a_returned_id_outside_the_pool(bad, b, at, spare):
    """In one of 300 sequences that are cut back, few tokens and many (which a kernel of its own writes)."""
    lens = [(37 * i) % 60 + 100 for i in range(300)]
    s = State(lens, 20, 6000, 16, seed=b)
    was = s.rows[b][at]
    s.t["block_tables"][b, at] = bad
    before = {k: v.clone() for k, v in s.t.items()}
    new, keep = [3] * 300, [(11 * i) % 14 for i in range(300)]
    n = 900 + spare
    for _ in range(2):
        cu, pos, slots = s.call(new, n, keep)
        assert s.pool.check() == pa.PA_ERR_DEVICE_BOUNDS
        for k, v in s.t.items():
            top = s.num_free if k == "free_blocks" else None
            assert torch.equal(v[:top], before[k][:top]), k
        assert not bool(cu.any()) and not bool(pos.any()) and bool((slots == -1).all())
    s.t["block_tables"][b, at] = was                       # mended by the host: the step goes on as if nothing had been
    s.free = s.t["free_blocks"].tolist()                   # entries at and beyond num_free are left over
    got = s.call(new, n, keep)
    s.check(got, s.expect(new, n, keep))
    assert s.pool.check() == pa.PA_OK


def test_an_id_outside_the_pool_that_is_kept():
    """Not returned: flagged where its tokens are written, as ever, and the step goes on."""
    s = State([20, 40], 6, 12, 16)
    s.t["block_tables"][0, 0] = 12
    got = s.call([1, 0], 1, [20, 3])
    s.rows[0][0] = 12
    s.check(got, s.expect([1, 0], 1, [20, 3]))
    assert s.pool.check() == pa.PA_OK
