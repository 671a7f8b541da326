"""prefill_packed (pa_prefill_packed) against the definition in 64 bits.

Tolerance, element by element, with h = eps / 2 of the type: the output is rounded once (h |out|); the
weights are rounded once to the type before the product with V (h sum p|v|); scores are fp32 sums of up
to 128 products: 128 2^-24 sum|q k| scale, at most 2^-13 for these inputs, in the weight and in the
normaliser (2^-12 sum p|v|, the exponential's own error far below).
"""
import math

import pytest
import torch

from paged_kv_cache_223_gb300 import pagedattn as pa
from serving_reference import packed_attention

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def make(seed, new, old, hq, hkv, d, dt, bs=16, spare_rows=0, first=0, nan_slots=True, qs=1.5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    lens = [a + b for a, b in zip(new, old)]
    blocks = [(x + bs - 1) // bs for x in lens]
    nb, stride = sum(blocks) + 2, max(blocks + [1]) + 1
    kc = torch.randn(nb, hkv, bs, d, generator=g, device=DEV).to(dt)
    vc = (torch.randn(nb, hkv, bs, d, generator=g, device=DEV) + 0.25).to(dt)
    ids = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    tables = torch.full((len(new), stride), 2 ** 31 - 1, dtype=torch.int32, device=DEV)   # never read past the context
    at = 0
    for b, m in enumerate(blocks):
        tables[b, :m] = ids[at:at + m]
        at += m
        if nan_slots and lens[b] % bs:
            kc[tables[b, m - 1].long(), :, lens[b] % bs:] = math.nan
            vc[tables[b, m - 1].long(), :, lens[b] % bs:] = math.nan
    for b in ids[at:]:
        kc[b.long()] = math.nan
        vc[b.long()] = math.nan
    cu = [first]
    for x in new:
        cu.append(cu[-1] + x)
    q = (torch.randn(cu[-1] + spare_rows, hq, d, generator=g, device=DEV) * qs).to(dt)
    pool = pa.Pool(nb, bs, hkv, d, dt, max_seqs=max(1, len(new)), max_q_heads=hq, max_q_len=1,
                   max_context_len=stride * bs, k_cache=kc, v_cache=vc)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    return pool, q, t(cu), tables, t(lens), 1.0 / math.sqrt(d)


def close(out, ref, mag, what=""):
    h = torch.finfo(out.dtype).eps / 2
    tol = ref.abs() * h + mag * (h * 1.01 + 2.0 ** -12) + 1e-6
    err = (out.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} outside, worst by {float((err - tol)[bad].max()):.3g}"


def check(pool, q, cu, tables, lens, scale, out=None, what=""):
    given = out
    out = pool.prefill_packed(q, cu, tables, lens, scale, out=out)
    assert pool.check() == pa.PA_OK
    ref, mag = packed_attention(q, pool.k_cache, pool.v_cache, cu.tolist(), tables, lens.tolist(), scale)
    lo, hi = int(cu[0]), int(cu[-1])
    close(out[lo:hi], ref[lo:hi], mag[lo:hi], what)
    return out if given is None else given


BF, FP = torch.bfloat16, torch.float16
CASES = [
    # new, old, hq, hkv, d, dtype, bs
    ([1], [0], 8, 2, 128, BF, 16),
    ([1], [0], 4, 4, 64, FP, 32),
    ([77], [0], 32, 8, 128, BF, 16),
    ([2, 0, 1, 300, 0], [0, 0, 500, 0, 20], 32, 8, 128, FP, 16),
    ([1, 17, 128, 129, 64, 63], [0, 0, 0, 0, 0, 0], 16, 4, 128, BF, 16),
    ([130, 5, 257, 31], [3, 1000, 255, 129], 64, 8, 128, BF, 32),
    ([200, 1, 90], [0, 77, 13], 8, 8, 64, FP, 16),
    ([100, 300], [0, 60], 6, 2, 128, FP, 16),              # G = 3: 42 positions a tile
    ([129, 40], [10, 0], 12, 1, 64, BF, 32),               # G = 12
    ([3, 70], [0, 5], 100, 1, 128, BF, 16),                # G = 100: one position a tile
    ([9, 5], [0, 130], 256, 2, 64, FP, 16),                # G = 128
    ([700], [0], 2, 1, 128, BF, 16),
    ([1500, 33, 600], [0, 2000, 100], 16, 4, 128, BF, 16),
    ([513, 1024], [0, 0], 4, 4, 64, BF, 16),
    ([9, 7, 14], [6000, 9001, 12345], 32, 8, 128, FP, 32),  # few rows behind long contexts
    ([1, 1, 1, 1], [5000, 1, 3000, 16000], 8, 8, 64, BF, 16),
    ([64], [30000], 8, 1, 128, BF, 16),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{i}-b{len(c[0])}-h{c[2]}.{c[3]}-d{c[4]}" for i, c in enumerate(CASES)])
def test_parity(case):
    new, old, hq, hkv, d, dt, bs = case
    check(*make(1 + CASES.index(case), new, old, hq, hkv, d, dt, bs))


def test_many_short_prompts():
    g = torch.Generator().manual_seed(3)
    new = torch.randint(0, 70, (300,), generator=g).tolist()
    old = torch.randint(0, 200, (300,), generator=g).tolist()
    check(*make(50, new, old, 8, 2, 128, BF))


def test_most_sequences():
    new = [1 if i % 3 else 2 for i in range(2048)]
    check(*make(51, new, [i % 50 for i in range(2048)], 4, 2, 64, FP, 16))


def test_rows_outside_the_sequences_are_left():
    pool, q, cu, tables, lens, scale = make(52, [33, 150], [0, 20], 8, 2, 128, BF, spare_rows=40, first=7)
    out = torch.full_like(q, 7.0)
    check(pool, q, cu, tables, lens, scale, out=out)
    assert bool((out[:7] == 7.0).all()) and bool((out[7 + 183:] == 7.0).all())


def test_peaked_and_flat_softmax():
    for qs in (0.0, 12.0):
        pool, q, cu, tables, lens, scale = make(53, [400, 90], [0, 900], 16, 4, 128, BF, qs=qs)
        out = pool.prefill_packed(q, cu, tables, lens, scale)
        ref, mag = packed_attention(q, pool.k_cache, pool.v_cache, cu.tolist(), tables, lens.tolist(), scale)
        # scores up to 12 |k|: their fp32 rounding, eight times that of the other cases
        h = torch.finfo(BF).eps / 2
        tol = ref.abs() * h + mag * (h * 1.01 + 2.0 ** -9) + 1e-6
        assert bool(((out.double() - ref).abs() <= tol).all())


def test_many_small_weights_beside_a_large_one():
    """One key takes nearly all the weight and has the value 0; the output is what 30000 keys of weight 2^-26 leave.
    Each of them is off by at most 2^-32 of the largest weight in fp16 (a relative half step in bf16)."""
    for dt in (FP, BF):
        pool, q, cu, tables, lens, scale = make(61, [3], [29997], 4, 2, 128, dt, nan_slots=False)
        bs = pool.geometry[2]
        pool.k_cache.zero_(), pool.v_cache.fill_(1.0), q.zero_()
        blk = int(tables[0, 0])
        q[:, :, 0] = 4.0
        pool.k_cache[blk, :, 5, 0] = 18.0 / (4.0 * scale)
        pool.v_cache[blk, :, 5] = 0.0
        out = pool.prefill_packed(q, cu, tables, lens, scale)
        ref, mag = packed_attention(q, pool.k_cache, pool.v_cache, cu.tolist(), tables, lens.tolist(), scale)
        assert 3e-4 < float(ref.min()) and float(ref.max()) < 6e-4
        h = torch.finfo(dt).eps / 2
        tol = ref * h + mag * (h * 1.01 + 2.0 ** -12) + 30000 * 2.0 ** -32
        assert bool(((out.double() - ref).abs() <= tol).all()), float((out.double() / ref).min())


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("heads", [(8, 2), (4, 4)])
def test_later_values_do_not_reach_earlier_rows(value, heads):
    """A key and a value of a later token hold no number: earlier rows do not see them, later rows do."""
    pool, q, cu, tables, lens, scale = make(54, [200, 40], [0, 100], heads[0], heads[1], 128, BF)
    bs = pool.geometry[2]
    for b, t in ((0, 131), (1, 120)):
        blk = int(tables[b, t // bs])
        pool.v_cache[blk, 0, t % bs, 5] = value
    out = pool.prefill_packed(q, cu, tables, lens, scale)
    ref, mag = packed_attention(q, pool.k_cache, pool.v_cache, cu.tolist(), tables, lens.tolist(), scale)
    fine = torch.isfinite(ref)
    assert not bool(fine.all()) and torch.equal(fine, torch.isfinite(out))
    close(out[fine], ref[fine], mag[fine])
    # a key without a number: rows at or behind it have no number, rows before it do not change
    before = out.clone()
    blk = int(tables[0, 150 // bs])
    pool.k_cache[blk, 1, 150 % bs, 3] = math.nan
    out = pool.prefill_packed(q, cu, tables, lens, scale)
    G = heads[0] // heads[1]
    assert bool(torch.isnan(out[150:200, G:2 * G]).all())
    assert torch.equal(out[:150, G:2 * G], before[:150, G:2 * G])


def test_determinism_and_other_caches():
    pool, q, cu, tables, lens, scale = make(55, [100, 40, 3], [0, 7000, 4000], 32, 8, 128, BF)
    a = pool.prefill_packed(q, cu, tables, lens, scale)
    for _ in range(3):
        assert torch.equal(a, pool.prefill_packed(q, cu, tables, lens, scale))
    k2, v2 = pool.k_cache.clone(), pool.v_cache.clone()
    pool.k_cache.zero_(), pool.v_cache.zero_()
    assert torch.equal(a, pool.prefill_packed(q, cu, tables, lens, scale, k_cache=k2, v_cache=v2))


def test_agrees_with_prefill_and_decode():
    """A batch with one length is pa_prefill's; single tokens are pa_decode's."""
    pool, q, cu, tables, lens, scale = make(56, [96, 96], [32, 500], 16, 4, 128, FP, nan_slots=False)
    a = pool.prefill_packed(q, cu, tables, lens, scale)
    tab = torch.where(tables < pool.geometry[0], tables, 0)
    b = pool.prefill(q.view(2, 96, 16, 128), tab, lens, scale).view(192, 16, 128)
    assert float((a.double() - b.double()).abs().max()) <= 4e-3
    pool, q, cu, tables, lens, scale = make(57, [1, 1, 1], [32, 500, 2000], 16, 4, 128, FP)
    a = pool.prefill_packed(q, cu, tables, lens, scale)
    b = pool.decode(q.view(3, 1, 16, 128), tables, lens, scale).view(3, 16, 128)
    assert float((a.double() - b.double()).abs().max()) <= 4e-3


def test_bad_tables_and_lengths_are_flagged():
    pool, q, cu, tables, lens, scale = make(58, [40, 50], [0, 100], 8, 2, 128, BF)
    ref = pool.prefill_packed(q, cu, tables, lens, scale)
    assert pool.check() == pa.PA_OK
    bad = tables.clone()
    bad[0, 1] = pool.geometry[0]
    out = pool.prefill_packed(q, cu, bad, lens, scale)
    assert pool.check() == pa.PA_ERR_DEVICE_BOUNDS and torch.equal(out[40:], ref[40:])
    short = lens.clone()
    short[0] = 20                                   # fewer tokens in the context than new ones
    out = pool.prefill_packed(q, cu, tables, short, scale)
    assert pool.check() == pa.PA_ERR_DEVICE_BOUNDS and torch.equal(out[40:], ref[40:])
    long = lens.clone()
    long[0] = tables.shape[1] * 16 + 1
    tab = torch.where(tables < pool.geometry[0], tables, 0)
    pool.prefill_packed(q, cu, tab, long, scale)
    assert pool.check() == pa.PA_ERR_DEVICE_BOUNDS
    wrong = cu.clone()
    wrong[2] = 1000                                 # past the rows of q
    pool.prefill_packed(q, wrong, tables, lens, scale)
    assert pool.check() == pa.PA_ERR_DEVICE_BOUNDS
    assert torch.equal(ref, pool.prefill_packed(q, cu, tables, lens, scale)) and pool.check() == pa.PA_OK


def test_refusals_on_the_host():
    pool, q, cu, tables, lens, scale = make(59, [40], [0], 8, 2, 128, BF)
    for bad in (lambda: pool.prefill_packed(q.view(40, -1), cu, tables, lens, scale),
                lambda: pool.prefill_packed(q, cu.long(), tables, lens, scale),
                lambda: pool.prefill_packed(q, cu[:0], tables, lens, scale),
                lambda: pool.prefill_packed(q.half(), cu, tables, lens, scale),
                lambda: pool.prefill_packed(q, torch.cat([cu, cu[1:]]), tables, lens, scale),
                lambda: pool.prefill_packed(q, cu, tables, lens[:0], scale),
                lambda: pool.prefill_packed(q, cu, tables, lens, scale, out=q[:8]),
                lambda: pool.prefill_packed(q[:, ::2], cu, tables, lens, scale)):
        with pytest.raises(ValueError):
            bad()
    both = torch.zeros(48, 8, 128, dtype=BF, device=DEV)
    for o in (q, both[8:]):                                        # out over q's own words, whole or in part
        with pytest.raises(pa.PagedAttnError):
            pool.prefill_packed(q if o is q else both[:40], cu, tables, lens, scale, out=o)
    wide = torch.zeros(1, 200, dtype=torch.int32, device=DEV)      # tables that may hold contexts worth cutting
    need = pool.packed_workspace(40, 1, 8, 200)
    assert need > 0 and pool.packed_workspace(40, 1, 8, tables.shape[1]) == 0
    for bad in (lambda: pool.prefill_packed(q[:, :5].contiguous(), cu, tables, lens, scale),
                lambda: pool.prefill_packed(q, cu, tables, lens, 0.0),
                lambda: pool.prefill_packed(q, cu, tables, lens, math.nan),
                lambda: pool.prefill_packed(q, cu, wide, lens, scale,
                                            workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV)),
                lambda: pool.packed_workspace(10, 5000, 8, 10)):
        with pytest.raises(pa.PagedAttnError):
            bad()
    fp8 = pa.Pool(8, 16, 2, 128, BF, max_context_len=128, kv_format=pa.PA_KV_FP8_E4M3)
    with pytest.raises(pa.PagedAttnError):
        fp8.prefill_packed(q, cu, tables, lens, scale)
    assert pool.prefill_packed(q[:0], cu[:1], tables, lens, scale).shape == (0, 8, 128)


def test_two_streams_at_once_and_graphs():
    """Two calls of one pool at the same time, and two captured ones replayed at the same time."""
    pool, q, cu, tables, lens, scale = make(60, [20, 9], [9000, 3000], 32, 8, 128, BF)
    ref = pool.prefill_packed(q, cu, tables, lens, scale)
    q2 = (q.float() * 0.5).to(BF)
    ref2 = pool.prefill_packed(q2, cu, tables, lens, scale)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a = pool.prefill_packed(q, cu, tables, lens, scale, stream=s1)
        b = pool.prefill_packed(q2, cu, tables, lens, scale, stream=s2)
        torch.cuda.synchronize()
        assert torch.equal(a, ref) and torch.equal(b, ref2)
    outs, graphs = [torch.empty_like(q), torch.empty_like(q)], []
    for x, o in zip((q, q2), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pool.prefill_packed(x, cu, tables, lens, scale, out=o)
        graphs.append(g)
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, (s1, s2)):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref2)
    # a captured call follows lengths that change between replays
    lens.sub_(5)
    graphs[0].replay()
    torch.cuda.synchronize()
    again, mag = packed_attention(q, pool.k_cache, pool.v_cache, cu.tolist(), tables, lens.tolist(), scale)
    close(outs[0], again, mag)
