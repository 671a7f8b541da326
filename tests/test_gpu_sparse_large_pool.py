"""The sparse decode step on pools whose caches and bounds lie beyond what 32 bits address: the results are those of a
small pool that holds the same blocks, bit for bit."""
import math

import pytest
import torch

from paged_kv_cache_223_gb300 import pagedattn as pa

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
HQ, HKV, D, BS, BLOCKS = 8, 2, 128, 16, 50


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def make(nb, dt, fp8):
    return pa.Pool(nb, BS, HKV, D, dt, max_seqs=2, max_q_heads=HQ, max_context_len=512,
                   kv_format=pa.PA_KV_FP8_E4M3 if fp8 else pa.PA_KV_16BIT)


def blocks_of(pool, cache):
    """Codes (or values) and scales of a cache, by blocks."""
    if cache.dtype != torch.uint8:
        return [cache]
    codes, scales = cache.split([pool.geometry[0] * HKV * BS * D, pool.geometry[0] * HKV * BS * 4])
    return [codes.view(-1, HKV, BS, D), scales.view(torch.float32).view(-1, HKV, BS)]


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


# 16-bit: 2^20 blocks of 8 KB, 8.6 GB a cache. FP8: 2^22 blocks of 4224 bytes, 17.7 GB a cache, bounds of 2.2 GB.
@pytest.mark.parametrize("dt,fp8,nb", [(torch.bfloat16, False, 2 ** 20 + 50), (torch.float16, True, 2 ** 22 + 50)])
def test_large_pools(dt, fp8, nb):
    torch.manual_seed(11)
    small, large = make(BLOCKS, dt, fp8), make(nb, dt, fp8)
    assert large.k_cache.numel() * large.k_cache.element_size() > 2 ** 32 and (not fp8 or large.bounds_size() > 2 ** 31)
    ids = torch.cat([torch.arange(nb - 30, nb, device=DEV), torch.arange(20, device=DEV)])[torch.randperm(BLOCKS, device=DEV)]
    for name in ("k_cache", "v_cache"):
        for i, (a, b) in enumerate(zip(blocks_of(small, getattr(small, name)), blocks_of(large, getattr(large, name)))):
            if not fp8:
                a.normal_()
            elif i == 0:
                a.copy_(torch.randint(0, 0x60, a.shape, device=DEV) + 0x80 * torch.randint(0, 2, a.shape, device=DEV))
            else:
                a.copy_(torch.rand(a.shape, device=DEV) * 0.1 + 0.01)
            b[ids] = a
    lens, cu, q = i32([400, 237]), i32([0, 400, 637]), torch.randn(2, 3, HQ, D, device=DEV).to(dt)
    order = torch.arange(BLOCKS, device=DEV).view(2, -1)
    results = []
    for pool, tables in ((small, order), (large, ids[order])):
        tables, bounds = tables.to(torch.int32).contiguous(), pool.new_bounds()
        pool.key_bounds(bounds, cu, tables, lens, 637)
        nb_ = pool.geometry[0]
        codes, steps = bounds[:nb_ * HKV * 2 * D].view(nb_, -1), bounds[nb_ * HKV * 2 * D:].view(nb_, -1)
        sel = pool.select_blocks(q, bounds, tables, lens, 9)
        out = pool.decode_selected(q, sel, tables, lens, 1 / math.sqrt(D))
        at = tables.long().flatten()
        results.append((codes[at], steps[at], sel, out.view(torch.int16)))
        assert pool.check() == pa.PA_OK
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert bool(results[0][0].any())
    # tables: blocks taken from the end of the pool, their slots
    free, num, row, n = torch.arange(nb, dtype=torch.int32, device=DEV), i32([nb]), i32([[-1] * 4]), i32([0])
    _, pos, slots = large.step_tables(i32([50]), n, row, free, num, 50)
    assert row.tolist() == [[nb - 1, nb - 2, nb - 3, nb - 4]] and num.tolist() == [nb - 4]
    assert slots.tolist() == [(nb - 1 - t // BS) * BS + t % BS for t in range(50)] and large.check() == pa.PA_OK
