"""Counts and scales of the sparse decode step's calls at the ends of what the C calls' types hold."""
import pytest
import torch

from paged_kv_cache_223_gb300 import pagedattn as pa

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.fixture(scope="module")
def step():
    pool = pa.Pool(8, 16, 2, 64, torch.float16, max_seqs=1, max_q_heads=4, max_context_len=128)
    pool.k_cache.normal_()
    pool.v_cache.normal_()
    return pool, torch.zeros(1, 1, 4, 64, dtype=torch.float16, device=DEV), i32([[3, 1, 2, 0]]), i32([64])


@pytest.mark.parametrize("n", [2 ** 32 + 4, 2 ** 31, -2 ** 31 - 1])
def test_counts_beyond_32_bits_are_refused(step, n):
    pool, q, tables, lens = step
    bounds, one = pool.new_bounds(), torch.zeros(0, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="num_tokens must fit"):
        pool.step_tables(i32([0]), lens, tables, torch.zeros(8, dtype=torch.int32, device=DEV), i32([0]), n, positions=one)
    with pytest.raises(ValueError, match="num_tokens must fit"):
        pool.key_bounds(bounds, i32([0, 4]), tables, lens, n)
    for kw in ("budget", "num_first", "num_last"):
        with pytest.raises(ValueError, match=kw + " must fit"):
            pool.select_blocks(q, bounds, tables, lens, **{**dict(budget=4), kw: n})
    assert pool.check() == pa.PA_OK and not bool(bounds.any()) and lens.tolist() == [64]


@pytest.mark.parametrize("scale", [2.2e38, -2.2e38, 2.5e38, 3.4e38, -3.4e38])
def test_scales_near_the_largest_number(step, scale):
    """Scores of 0 whatever the scale: the mean of V, as long as scale times log2(e) is a number (log2(e) 2.2e38 = 3.17e38,
    2.5e38: 3.61e38, beyond 3.40e38), else a refusal."""
    pool, q, tables, lens = step
    sel = i32([[[0, 1, 2, 3], [0, 1, 2, 3]]])
    if abs(scale) > 2.3e38:
        with pytest.raises(pa.PagedAttnError):
            pool.decode_selected(q, sel, tables, lens, scale)
        return
    out = pool.decode_selected(q, sel, tables, lens, scale)
    v = pool.v_cache[tables[0].long()].double().mean((0, 2))           # [2, 64]
    # the output's rounding, the weights' 22 bits, and 64 sums and their joining in fp32
    tol = torch.finfo(torch.float16).eps / 2 * float(v.abs().max()) + 2 ** -16 * float(pool.v_cache.abs().max())
    assert float((out[0, 0].view(2, 2, 64).double() - v[:, None]).abs().max()) <= tol
    assert pool.check() == pa.PA_OK
