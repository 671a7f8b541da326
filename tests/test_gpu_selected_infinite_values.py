"""decode_selected with infinities and NaN among the values that every row sees: an output dimension is what a softmax gives,
the infinity where the weighted sum holds one, NaN where it holds both or a NaN; the other dimensions keep their tolerance."""
import math

import pytest
import torch

from test_gpu_decode_selected import i32, make, pick
from test_gpu_selected_bits import definition, run

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.mark.parametrize("dt,d,hq,hkv,q_len", [(torch.float16, 128, 8, 2, 1), (torch.bfloat16, 128, 8, 2, 1),
                                               (torch.bfloat16, 64, 16, 2, 2), (torch.float16, 128, 12, 2, 4),
                                               (torch.bfloat16, 128, 16, 1, 2)])
def test_infinities_and_nan_that_every_row_sees(dt, d, hq, hkv, q_len):
    lens = [700, 90, 33]
    pool, tables, q = make(lens, hq, hkv, d, dt, 16, q_len, seed=d + hq)
    sel = pick(lens, hkv, 16, 40, 5)
    v = pool.v_cache
    first, later, last = (int(tables[0, j]) for j in (0, 20, 43))
    v[first, 0, 3, 5] = math.inf
    v[first, 0, 7, 6] = -math.inf
    v[later, 0, 0, 5] = math.inf                           # two of one sign
    v[later, 0, 1, 6] = math.inf                           # one of each: NaN
    v[later, 0, 2, 9] = math.nan
    v[last, hkv - 1, 2, 11] = -math.inf                    # beside tokens that not every row sees
    v[int(tables[1, 0]), 0, :, 2] = math.inf               # a whole block
    for cache in (pool.k_cache, v):                        # behind the context, where the tiles are looked at again
        cache[last, :, 12:] = math.nan
    if q_len > 1:
        v[last, 0, 11] = math.inf                          # the newest draft's, beside them
    sel[0, :, :3] = i32([0, 20, 43])
    sel[0, :, 3:] = i32([j for j in range(44) if j not in (0, 20, 43)][:37])
    out = definition(pool, q, sel, tables, lens, 0.1)[0]
    assert bool(out.isinf().any()) and bool(out.isnan().any()) and bool(out.isfinite().any())
    run(pool, tables, q, lens, sel, 0.1)


@pytest.mark.parametrize("hq", [2, 8, 16, 24, 32])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_fp8_scales_that_are_no_numbers(dt, hq):
    """A token of an infinite V scale: infinity by its code's sign (its codes are no zeros), a NaN code or scale: NaN."""
    lens = [600, 100]
    pool, tables, q = make(lens, hq, 2, 128, dt, 16, 2, fp8=True, seed=4)
    sel = pick(lens, 2, 16, 38, 6)
    nb, hkv, bs, d = pool.geometry
    codes = pool.v_cache[:nb * hkv * bs * d].view(nb, hkv, bs, d)
    scales = pool.v_cache[nb * hkv * bs * d:].view(torch.float32).view(nb, hkv, bs)
    codes[(codes & 0x7F) == 0] = 0x08
    a, b = int(tables[0, 17]), int(tables[1, 2])
    scales[a, 0, 4] = math.inf
    codes[a, 1, 9, 77] = 0x7F
    scales[b, 1, 0] = math.nan
    last = int(tables[1, 6])                               # tokens 96 to 99, the last of them a draft of one row
    scales[last, :, 4:], codes[last, :, 5:] = math.nan, 0x7F
    scales[last, 0, 3] = math.inf
    out = definition(pool, q, sel, tables, lens, 0.1)[0]
    assert bool(out.isinf().any()) and bool(out.isnan().any()) and bool(out.isfinite().any())
    run(pool, tables, q, lens, sel, 0.1)


@pytest.mark.parametrize("fp8", [False, True])
def test_the_same_with_many_tiles_a_warp(fp8):
    """Lists of many tiles: copies are in flight again behind the first look at the values."""
    lens = [6000]
    pool, tables, q = make(lens, 8, 1, 128, torch.float16, 16, 1, fp8=fp8, seed=8)
    sel = torch.arange(375, dtype=torch.int32, device=DEV).view(1, 1, -1).contiguous()
    nb, hkv, bs, d = pool.geometry
    for j, t in ((3, 2), (200, 9), (374, 15)):
        if fp8:
            pool.v_cache[(int(tables[0, j]) * bs + t) * d + 12 + t] = 0x7F
        else:
            pool.v_cache[int(tables[0, j]), 0, t, 12 + t] = math.inf
    first = run(pool, tables, q, lens, sel, 0.1)
    assert torch.equal(run(pool, tables, q, lens, sel, 0.1).view(torch.int16), first.view(torch.int16))
