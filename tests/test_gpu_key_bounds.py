"""key_bounds (pa_key_bounds) against its definition: a largest and a smallest key, a power of two, one rounding. Equal."""
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_223_gb300 import pagedattn as pa
from sparse_reference import bounds_of, ceil_div

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def parts(pool, bounds):
    nb, hkv, _, d = pool.geometry
    n = nb * hkv * 2 * d
    return bounds[:n].view(torch.int8).view(nb, hkv, 2, d), bounds[n:].view(torch.float32).view(nb, hkv)


def keys_of(pool, k_cache=None):
    """The cache's values as the operators see them: numbers of 32 bits."""
    nb, hkv, bs, d = pool.geometry
    k = pool.k_cache if k_cache is None else k_cache
    if pool.kv_format == pa.PA_KV_FP8_E4M3:
        n = nb * hkv * bs * d
        return k[:n].view(torch.float8_e4m3fn).float().view(nb, hkv, bs, d) * k[n:].view(torch.float32).view(nb, hkv, bs, 1)
    return k.float()


def expected(pool, before, cu, rows, lens, k_cache=None):
    """(codes, steps) as numpy arrays: what was there, with the touched blocks made anew."""
    codes, steps = (x.cpu().numpy().copy() for x in parts(pool, before))
    keys = keys_of(pool, k_cache).double().cpu().numpy()
    bs = pool.geometry[2]
    for b, n in enumerate(lens):
        new = cu[b + 1] - cu[b]
        for j in range((n - new) // bs, ceil_div(n, bs)) if new else ():
            for h in range(pool.geometry[1]):
                codes[rows[b][j], h], steps[rows[b][j], h] = bounds_of(keys[rows[b][j], h, :n - j * bs])
    return codes, steps


def check(pool, bounds, want):
    codes, steps = (x.cpu().numpy() for x in parts(pool, bounds))
    assert np.array_equal(steps, want[1].astype(np.float32)) and np.array_equal(codes, want[0])


def make(lens, hkv, d, dt, bs, fp8=False, seed=0, spare=2, small=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    nb = sum(ceil_div(n, bs) for n in lens) + spare
    pool = pa.Pool(nb, bs, hkv, d, dt, max_seqs=1, max_context_len=512,
                   kv_format=pa.PA_KV_FP8_E4M3 if fp8 else pa.PA_KV_16BIT)
    if fp8:
        n = nb * hkv * bs * d
        pool.k_cache[:n] = torch.randn(n, generator=g, device=DEV).mul_(100).to(torch.float8_e4m3fn).view(torch.uint8)
        pool.k_cache[n:].view(torch.float32).copy_(torch.rand(n // d, generator=g, device=DEV) * 0.02 + 1e-4)
    else:
        x = torch.randn(nb, hkv, bs, d, generator=g, device=DEV)
        if small:                                        # every size there is, subnormal ones among them
            x *= torch.exp2(torch.randint(-20, 12, (nb, hkv, 1, 1), generator=g, device=DEV).float() * (1 if dt == torch.float16 else 6))
        pool.k_cache.copy_(x)
    ids = torch.randperm(nb, generator=g, device=DEV).tolist()
    rows, stride = [], max([1] + [ceil_div(n, bs) for n in lens])
    for n in lens:
        k = ceil_div(n, bs)
        rows.append(ids[:k] + [-1] * (stride - k))
        ids = ids[k:]
    bounds = torch.randint(0, 256, (pool.bounds_size(),), generator=g, device=DEV, dtype=torch.uint8)
    parts(pool, bounds)[1].fill_(3.0)
    return pool, rows, bounds


def run(pool, rows, bounds, new, lens, pad=0):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    want = expected(pool, bounds, cu, rows, lens)
    pool.key_bounds(bounds, i32(cu), i32(rows), i32(lens), cu[-1] + pad)
    check(pool, bounds, want)
    return want


@pytest.mark.parametrize("lens,new,hkv,d,dt,bs,fp8", [
    ([1], [1], 1, 64, torch.float16, 16, False),
    ([17], [1], 8, 128, torch.bfloat16, 16, False),
    ([33, 32, 31, 1], [1, 32, 16, 0], 2, 128, torch.float16, 32, False),
    ([300, 7, 64, 65], [299, 7, 1, 2], 3, 64, torch.bfloat16, 16, False),
    ([200, 201, 5], [40, 201, 1], 4, 128, torch.bfloat16, 32, True),
    ([16, 47], [16, 31], 1, 128, torch.float16, 16, True),
    ([2000, 1], [2000, 1], 8, 128, torch.bfloat16, 16, False),
    ([(7 * i) % 50 + 1 for i in range(300)], [(i % 3) and 1 for i in range(300)], 2, 64, torch.float16, 16, False),
])
def test_bounds(lens, new, hkv, d, dt, bs, fp8):
    pool, rows, bounds = make(lens, hkv, d, dt, bs, fp8, seed=len(lens) + d)
    run(pool, rows, bounds, new, lens, pad=3)
    assert pool.check() == pa.PA_OK


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_sizes_of_every_kind(dt):
    pool, rows, bounds = make([700], 2, 64, dt, 16, small=True)
    pool.k_cache[rows[0][0]] = 0.0                       # a step of 0
    pool.k_cache[rows[0][1], :, :, 1:] = 0.0
    pool.k_cache[rows[0][2]] = -0.0
    for i, x in enumerate((127.0, 127.5, 63.5, 64.0, -127.0, 254.0)):
        pool.k_cache[rows[0][3 + i]] = 1.0
        pool.k_cache[rows[0][3 + i], :, 3, 5] = x
    big, tiny = torch.finfo(dt).max, torch.finfo(dt).smallest_normal * torch.finfo(dt).eps
    pool.k_cache[rows[0][9], 0, 2, 3] = -big
    pool.k_cache[rows[0][10]] = tiny
    run(pool, rows, bounds, [700], [700])
    assert pool.check() == pa.PA_OK


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("x", [math.nan, math.inf, -math.inf])
def test_no_numbers(fp8, x):
    """In a token that counts: an infinite step. Behind the context, and in blocks beside: nothing."""
    pool, rows, bounds = make([40, 40], 2, 128, torch.float16, 16, fp8)
    nb, hkv, bs, d = pool.geometry

    def put(block, h, t):
        if fp8:                                           # codes have NaN only, scales may be anything
            i = (block * hkv + h) * bs + t
            if math.isnan(x):
                pool.k_cache[i * d + 7] = 0x7F
            else:
                pool.k_cache[nb * hkv * bs * d:].view(torch.float32)[i] = x
                pool.k_cache[i * d:(i + 1) * d] = 0x38
        else:
            pool.k_cache[block, h, t, 7] = x
    put(rows[0][1], 1, 3)
    put(rows[0][2], 0, 7)                                 # token 39: the last one
    put(rows[1][2], 0, 8)                                 # token 40: behind the context
    want = run(pool, rows, bounds, [40, 40], [40, 40])
    assert want[1][rows[0][1], 1] == math.inf and want[1][rows[0][2], 0] == math.inf
    assert np.isfinite(np.delete(want[1].reshape(-1), [rows[0][1] * 2 + 1, rows[0][2] * 2])).all()
    assert pool.check() == pa.PA_OK


def test_fp8_subnormal_scales():
    pool, rows, bounds = make([60], 1, 128, torch.bfloat16, 32, True)
    n = pool.geometry[0] * 32 * 128
    pool.k_cache[n:].view(torch.float32).mul_(2.0 ** -139)
    run(pool, rows, bounds, [60], [60])


def test_another_cache_and_a_captured_step():
    pool, rows, bounds = make([50, 3], 2, 64, torch.bfloat16, 16)
    other = torch.randn_like(pool.k_cache)
    cu, lens = i32([0, 1, 4]), i32([50, 3])
    want = expected(pool, bounds, [0, 1, 4], rows, [50, 3], other)
    pool.key_bounds(bounds, cu, i32(rows), lens, 4, k_cache=other)
    check(pool, bounds, want)
    tables = i32(rows)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pool.key_bounds(bounds, cu, tables, lens, 4)
    for n in (49, 17, 33):
        lens[0] = n
        want = expected(pool, bounds, [0, 1, 4], rows, [n, 3])
        g.replay()
        check(pool, bounds, want)
    assert pool.check() == pa.PA_OK


@pytest.mark.parametrize("what", ["cu_down", "cu_high", "cu_negative", "short", "long", "id"])
def test_what_does_not_fit_is_skipped(what):
    pool, rows, bounds = make([40, 40, 40], 2, 64, torch.float16, 16)
    cu, lens, bad = [0, 5, 10, 15], [40, 40, 40], [1]
    if what == "cu_down":
        cu = [0, 5, 4, 15]
    elif what == "cu_high":
        cu, bad = [0, 5, 10, 16], [2]
    elif what == "cu_negative":
        cu, bad = [-1, 5, 10, 15], [0]
    elif what == "short":
        lens[1] = 4
    elif what == "long":
        lens[1] = 49
    elif what == "id":
        rows[1][2] = pool.geometry[0]
    fit_cu = [0, 5, 10, 15] if what != "cu_down" else [0, 5, 5, 16]
    want_rows = [r if i not in bad else None for i, r in enumerate(rows)]
    codes, steps = (x.cpu().numpy().copy() for x in parts(pool, bounds))
    keys = keys_of(pool).double().cpu().numpy()
    for b in range(3):
        if want_rows[b] is None and what != "id":
            continue
        new = fit_cu[b + 1] - fit_cu[b]
        for j in range((40 - new) // 16, 3):
            if rows[b][j] < pool.geometry[0]:
                for h in range(2):
                    codes[rows[b][j], h], steps[rows[b][j], h] = bounds_of(keys[rows[b][j], h, :40 - j * 16])
    pool.key_bounds(bounds, i32(cu), i32(rows), i32(lens), 15)
    assert pool.check() == pa.PA_ERR_DEVICE_BOUNDS
    check(pool, bounds, (codes, steps))


def test_sequences_that_share_rows_have_no_more_work_than_a_call():
    """Every other sequence of 2000 names all rows: flagged, nothing done."""
    pool, rows, bounds = make([1000], 1, 64, torch.float16, 16)
    before, n = bounds.clone(), 2000
    pool.key_bounds(bounds, i32([0, 1000] * (n // 2) + [0]), i32(rows).repeat(n, 1), i32([1000] * n), 1000)
    assert pool.check() == pa.PA_ERR_DEVICE_BOUNDS and torch.equal(bounds, before)


def test_refusals():
    pool, rows, bounds = make([40], 2, 64, torch.float16, 16)
    L, cu, tables, lens = pa._sparse_lib(), i32([0, 1]), i32(rows), i32([40])
    good = [pool.handle, None, cu.data_ptr(), tables.data_ptr(), 3, lens.data_ptr(), 1, 1, bounds.data_ptr(), None]
    before = bounds.clone()
    for i, v in ((2, None), (3, None), (4, 0), (5, None), (6, -1), (7, -1), (8, None), (8, bounds.data_ptr() + 4),
                 (8, pool.k_cache.data_ptr() + 16), (1, pool.k_cache.data_ptr() + 2), (2, cu.data_ptr() + 1),
                 (2, bounds.data_ptr()), (3, bounds.data_ptr() + 16)):
        a = list(good)
        a[i] = v
        assert L.pa_key_bounds(*a) == pa.PA_ERR_INVALID_ARG, (i, v)
    a = list(good)
    a[7] = 8193
    assert L.pa_key_bounds(*a) == pa.PA_ERR_UNSUPPORTED
    for i in (6, 7):                                      # nothing to do
        a = list(good)
        a[i] = 0
        assert L.pa_key_bounds(*a) == pa.PA_OK
    for kw in (dict(bounds=bounds[:-1]), dict(bounds=bounds.view(torch.int8)), dict(cu_q=cu.long()), dict(cu_q=cu[:0]),
               dict(block_tables=tables[:0]), dict(context_lens=lens.cpu()), dict(k_cache=pool.k_cache.float())):
        with pytest.raises(ValueError):
            pool.key_bounds(**{**dict(bounds=bounds, cu_q=cu, block_tables=tables, context_lens=lens, num_tokens=1), **kw})
    assert torch.equal(bounds, before) and pool.check() == pa.PA_OK
