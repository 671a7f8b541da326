"""decode_selected (pa_decode_selected) against attention over the listed blocks in 64 bits.

Tolerance of an output, relative to sum p |v| but for the last rounding (eps / 2 of the value):
- weights go into the product as two parts of 16 bits (2^-16 for bf16, less for fp16), in FP8 pools as one of fp16 (2^-11);
  parts of fp16 below 2^-14 lose up to 2^-25 each, of a sum of weights that is at least 1 (FP8: times the V scale, in
  units of a power of two not above the largest scale): N 2^-25 max |v|;
- a score is a fp32 sum of products whose sizes add up to `big` (in units of e): 2^-20 big, twice (score and reference);
- exponentials and sums of 32 bits: 2^-20;
- a product's accumulator may drop the last bit of each of its N / 16 additions: N 2^-26.
"""
import math

import pytest
import torch

from paged_kv_cache_223_gb300 import pagedattn as pa
from sparse_reference import attend, ceil_div

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def make(lens, hq, hkv, d, dt, bs, q_len=1, fp8=False, seed=0, spare=2, vscale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    blocks = [ceil_div(n, bs) for n in lens]
    nb = sum(blocks) + spare
    pool = pa.Pool(nb, bs, hkv, d, dt, max_seqs=1, max_q_heads=hq, max_context_len=512,
                   kv_format=pa.PA_KV_FP8_E4M3 if fp8 else pa.PA_KV_16BIT)
    for i, c in enumerate((pool.k_cache, pool.v_cache)):
        x = torch.randn(nb, hkv, bs, d, generator=g, device=DEV) * (vscale if i else 1.0)
        if fp8:
            s = x.abs().amax(-1) / 448.0
            c.copy_(torch.cat([(x / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(-1),
                               s.view(-1).view(torch.uint8)]))
        else:
            c.copy_(x)
    ids = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    tables, at = torch.full((len(lens), max([1] + blocks)), -1, dtype=torch.int32, device=DEV), 0
    for i, k in enumerate(blocks):
        tables[i, :k] = ids[at:at + k]
        at += k
    q = (torch.randn(len(lens), q_len, hq, d, generator=g, device=DEV) * 1.2).to(dt)
    return pool, tables, q


def pick(lens, hkv, bs, budget, seed, order="ascending"):
    """Lists that hold the last block and others anywhere; -1 where the context has fewer."""
    g = torch.Generator().manual_seed(seed)
    out = torch.full((len(lens), hkv, budget), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        k = ceil_div(n, bs)
        for h in range(hkv):
            if k:
                some = torch.randperm(k - 1, generator=g)[:budget - 1].tolist() + [k - 1]
                some = sorted(some) if order == "ascending" else some
                if order == "holes":
                    at = torch.randperm(budget, generator=g)[:len(some)]
                    out[b, h, at] = torch.tensor(some, dtype=torch.int32)
                else:
                    out[b, h, :len(some)] = torch.tensor(some, dtype=torch.int32)
    return out.to(DEV)


def reader(pool, cache, tables):
    nb, hkv, bs, d = pool.geometry
    if pool.kv_format == pa.PA_KV_FP8_E4M3:
        n = nb * hkv * bs * d
        x = cache[:n].view(torch.float8_e4m3fn).double().view(nb, hkv, bs, d) * cache[n:].view(torch.float32).double().view(nb, hkv, bs, 1)
    else:
        x = cache.double()
    return lambda b, h, j: x[tables[b, j].long(), h]


def reference(pool, q, selected, tables, lens, scale, k_cache=None, v_cache=None):
    return attend(q, reader(pool, pool.k_cache if k_cache is None else k_cache, tables),
                  reader(pool, pool.v_cache if v_cache is None else v_cache, tables), selected, lens, scale)


def close(got, ref, selected, bs, fp8, vmax):
    out, mag, big = ref
    dt = got.dtype
    n = selected.shape[-1] * bs
    rel = (2.0 ** -11 if fp8 else 2.0 ** -16) + big[..., None] * 2.0 ** -19 + 2.0 ** -20 + n * 2.0 ** -26
    tol = out.abs() * torch.finfo(dt).eps / 2 + mag * rel + (n * 2.0 ** -25 * vmax if fp8 or dt == torch.float16 else 0)
    tol = tol + torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2
    err = (got.double() - out).abs()
    assert bool((err <= tol).all()), f"{int((~(err <= tol)).sum())} outside, worst {float((err - tol).max()):.3g}"


def run(pool, tables, q, lens, selected, scale=None, vmax=None):
    d, bs = pool.geometry[3], pool.geometry[2]
    scale = 1 / math.sqrt(d) if scale is None else scale
    got = pool.decode_selected(q, selected, tables, i32(lens), scale)
    fp8 = pool.kv_format == pa.PA_KV_FP8_E4M3
    vmax = vmax or (6.0 if fp8 else float(pool.v_cache.float().nan_to_num(0.0, 0.0, 0.0).abs().max()))
    close(got, reference(pool, q, selected, tables, lens, scale), selected, bs, fp8, vmax)
    return got


CASES = [
    # lens, hq, hkv, d, dtype, bs, q_len, budget
    ([1], 1, 1, 64, torch.float16, 16, 1, 1),
    ([16], 8, 1, 128, torch.bfloat16, 16, 1, 3),
    ([500, 17, 33, 2], 32, 8, 128, torch.bfloat16, 16, 1, 9),
    ([1000], 16, 16, 64, torch.float16, 32, 1, 20),
    ([700, 90], 12, 4, 128, torch.float16, 32, 3, 7),
    ([300, 299, 8], 8, 4, 64, torch.bfloat16, 16, 8, 12),
    ([1500, 31], 64, 8, 128, torch.float16, 16, 2, 40),
    ([400, 5], 20, 4, 128, torch.bfloat16, 16, 5, 11),         # 25 rows
    ([900, 65], 32, 1, 128, torch.bfloat16, 32, 1, 16),        # a group of 32
    ([640], 16, 2, 64, torch.float16, 16, 4, 30),
    ([5000], 8, 2, 128, torch.bfloat16, 16, 1, 300),
    ([260] * 33, 16, 8, 128, torch.float16, 16, 1, 8),
]


@pytest.mark.parametrize("order", ["ascending", "any", "holes"])
@pytest.mark.parametrize("lens,hq,hkv,d,dt,bs,q_len,budget", CASES)
def test_attention(lens, hq, hkv, d, dt, bs, q_len, budget, order):
    pool, tables, q = make(lens, hq, hkv, d, dt, bs, q_len, seed=budget)
    run(pool, tables, q, lens, pick(lens, hkv, bs, budget, 1, order))
    assert pool.check() == pa.PA_OK


@pytest.mark.parametrize("lens,hq,hkv,dt,bs,q_len,budget", [([1], 4, 4, torch.float16, 16, 1, 2),
                                                            ([500, 33, 64], 32, 8, torch.bfloat16, 32, 1, 6),
                                                            ([700, 90, 6], 8, 2, torch.float16, 16, 6, 20),
                                                            ([300, 47], 16, 2, torch.bfloat16, 16, 4, 10),
                                                            ([4000], 8, 1, torch.float16, 16, 2, 200)])
def test_fp8_pools(lens, hq, hkv, dt, bs, q_len, budget):
    pool, tables, q = make(lens, hq, hkv, 128, dt, bs, q_len, fp8=True, seed=budget)
    run(pool, tables, q, lens, pick(lens, hkv, bs, budget, 2))
    assert pool.check() == pa.PA_OK


@pytest.mark.parametrize("vscale", [1e-6, 1e4])
def test_fp8_values_of_any_size(vscale):
    """V scales far below and above fp16's normal numbers; sizes that grow and shrink along the context."""
    lens = [600, 100]
    pool, tables, q = make(lens, 8, 2, 128, torch.bfloat16, 16, 2, fp8=True, vscale=vscale)
    sel = pick(lens, 2, 16, 30, 3)
    run(pool, tables, q, lens, sel, vmax=6 * vscale)
    n = pool.geometry[0] * 2 * 16
    grow = torch.exp2(torch.arange(n, device=DEV).float() % 37 - 18)
    pool.v_cache[n * 128:].view(torch.float32).mul_(grow)
    run(pool, tables, q, lens, sel, vmax=6 * vscale * 2 ** 18)
    assert pool.check() == pa.PA_OK


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_fp8_blocks_of_new_tokens_only(dt):
    """The only listed block holds tokens that not every row sees: no scale is common to the rows."""
    lens = [18, 33, 50, 17]
    pool, tables, q = make(lens, 8, 2, 128, dt, 16, 4, fp8=True, seed=9)
    sel = i32([[[1, -1], [1, 0]], [[2, -1], [-1, 2]], [[3, 0], [3, -1]], [[-1, 1], [1, -1]]])
    run(pool, tables, q, lens, sel)


def test_fp8_bf16_queries_beyond_fp16():
    lens = [300]
    pool, tables, q = make(lens, 8, 2, 128, torch.bfloat16, 16, 2, fp8=True)
    q[:, :, ::2] *= 2.0 ** 20
    n = pool.geometry[0] * 2 * 16 * 128
    pool.k_cache[n:].view(torch.float32).mul_(2.0 ** -16)
    run(pool, tables, q, lens, pick(lens, 2, 16, 8, 4))


def test_fp8_small_bf16_queries():
    """Queries below fp16's normal numbers against large keys."""
    lens = [300]
    pool, tables, q = make(lens, 8, 2, 128, torch.bfloat16, 16, 2, fp8=True)
    q *= 2.0 ** -22
    n = pool.geometry[0] * 2 * 16 * 128
    pool.k_cache[n:].view(torch.float32).mul_(2.0 ** 22)
    run(pool, tables, q, lens, pick(lens, 2, 16, 8, 4))
    q *= 2.0 ** -90
    pool.k_cache[n:].view(torch.float32).mul_(2.0 ** 90)
    run(pool, tables, q, lens, pick(lens, 2, 16, 8, 4))


def test_all_blocks_listed_is_decode():
    lens = [777, 64, 1]
    pool, tables, q = make(lens, 32, 8, 128, torch.bfloat16, 16)
    pool2 = pa.Pool(*[pool.geometry[i] for i in (0, 2, 1, 3)], torch.bfloat16, max_seqs=3, max_q_heads=32, max_context_len=1024,
                    k_cache=pool.k_cache, v_cache=pool.v_cache)
    sel = torch.arange(49, dtype=torch.int32, device=DEV).repeat(3, 8, 1)
    for b, n in enumerate(lens):
        sel[b][:, ceil_div(n, 16):] = -1
    dense = pool2.decode(q, tables, i32(lens), 0.1)
    sparse = run(pool, tables, q, lens, sel.contiguous(), scale=0.1)
    assert float((dense.double() - sparse.double()).abs().max()) <= 2 * torch.finfo(torch.bfloat16).eps * float(dense.abs().max())


def test_nothing_listed_and_nothing_seen():
    lens = [100, 0, 40, 40]
    pool, tables, q = make(lens, 8, 2, 64, torch.float16, 16, 5)
    sel = torch.full((4, 2, 4), -1, dtype=torch.int32, device=DEV)
    sel[0, 0, 2] = 6                                       # tokens 96..99: rows 0..3 see some, all of them 96 or more
    sel[2, 1, 0] = 2                                       # tokens 32..39, rows at 35..39
    sel[3, 0, 0] = -2 ** 31
    got = run(pool, tables, q, lens, sel)
    assert bool((got[1] == 0).all()) and bool((got[0, :, 4:] == 0).all()) and bool((got[3] == 0).all())
    assert bool((got[2, :, :4] == 0).all()) and pool.check() == pa.PA_OK
    sel[0, 0, 2] = -1
    sel[0, 0, 0] = 6
    lens[0] = 98                                           # rows at 93..97: three of them see nothing of 96..97
    got = run(pool, tables, q, lens, sel)
    assert bool((got[0, :3] == 0).all()) and bool((got[0, 3:, :4] != 0).any())


@pytest.mark.parametrize("fp8", [False, True])
def test_scores_of_minus_infinity(fp8):
    """Where some are, their tokens have no weight; where all are, a softmax has no value; where nothing is seen, zeros."""
    lens = [64, 64, 64]
    pool, tables, q = make(lens, 4, 1, 128, torch.float16, 16, 2, fp8=fp8)
    q[..., 0] = 1.0
    nb = pool.geometry[0]
    for block in (tables[0, 1], tables[1, 1], tables[1, 3]):
        i = int(block)
        if fp8:                                           # one dimension of -1, the others 0 with a NaN scale's stead: -inf
            pool.k_cache[nb * 16 * 128:].view(torch.float32)[i * 16:(i + 1) * 16] = 3e38
            pool.k_cache[i * 16 * 128:(i + 1) * 16 * 128] = 0
            pool.k_cache[i * 16 * 128:(i + 1) * 16 * 128].view(16, 128)[:, 0] = 0xFE      # -448
        else:
            pool.k_cache[i, 0, :, 0] = -math.inf
    sel = i32([[[1, 2]], [[1, 3]], [[-1, -1]]])
    got = pool.decode_selected(q, sel, tables, i32(lens), 1.0)
    ref = reference(pool, q, i32([[[2, -1]], [[-1, -1]], [[-1, -1]]]), tables, lens, 1.0)
    close(got[:1], [x[:1] for x in ref], sel, 16, fp8, 6.0)
    assert bool(torch.isnan(got[1]).all()) and bool((got[2] == 0).all())


def test_a_block_listed_twice_counts_twice():
    lens = [200]
    pool, tables, q = make(lens, 4, 1, 128, torch.float16, 16)
    sel = i32([[[3, 5, 3, 12, 3]]])
    run(pool, tables, q, lens, sel)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("x", [math.nan, math.inf])
def test_what_a_row_does_not_see_does_not_reach_it(fp8, x):
    """NaN and infinities behind the context, in blocks that are not listed, and in drafts that a row does not see."""
    lens = [70, 41]
    pool, tables, q = make(lens, 8, 2, 128, torch.float16, 16, 4, fp8=fp8, seed=5)
    nb, hkv, bs, d = pool.geometry
    n = nb * hkv * bs
    sel = i32([[[0, 3, 4], [1, 2, 4]], [[0, 2, -1], [2, 1, -1]]])
    clean = run(pool, tables, q, lens, sel)

    def put(block, t):
        for c in (pool.k_cache, pool.v_cache):
            if fp8:
                for h in range(hkv):
                    i = (block * hkv + h) * bs + t
                    c[i * d:(i + 1) * d] = 0x7F
                    c[n * d:].view(torch.float32)[i] = x
            else:
                c[block, :, t] = x
    for b, length in enumerate(lens):
        for t in range(length % bs, bs):
            put(int(tables[b, length // bs]), t)
    free = next(i for i in range(nb) if int((tables == i).sum()) == 0)
    for t in range(bs):
        put(free, t)
    assert torch.equal(run(pool, tables, q, lens, sel), clean)
    # the newest draft: its own row has no number, the rows before it keep theirs
    put(int(tables[0, 4]), 69 % bs)
    got = pool.decode_selected(q, sel, tables, i32(lens), 1 / math.sqrt(d))
    assert torch.equal(got[0, :3], clean[0, :3]) and torch.equal(got[1], clean[1])
    assert bool(torch.isnan(got[0, 3]).all()) if math.isnan(x) else not bool(torch.isfinite(got[0, 3]).all())
    assert pool.check() == pa.PA_OK


@pytest.mark.parametrize("what", ["beyond", "id", "negative id", "length", "negative", "short"])
def test_what_does_not_fit_is_flagged_and_skipped(what):
    lens = [150, 150]
    pool, tables, q = make(lens, 8, 2, 64, torch.bfloat16, 16, 2)
    sel = pick(lens, 2, 16, 6, 6)
    want, as_lens = sel.clone(), list(lens)
    dl = list(lens)
    if what == "beyond":
        sel[0, 0, 1], want[0, 0, 1] = 10, -1
    elif what in ("id", "negative id"):
        j = int(sel[0, 1, 1])
        tables[0, j] = pool.geometry[0] if what == "id" else -1
        want[0][want[0] == j] = -1
    elif what == "length":
        dl[0], as_lens[0] = 161, 160
    elif what == "negative":
        dl[0], as_lens[0], want[0] = -1, 0, -1
    elif what == "short":
        dl[0], as_lens[0] = 1, 1
        want[0][want[0] > 0] = -1
    got = pool.decode_selected(q, sel, tables, i32(dl), 0.125)
    assert pool.check() == pa.PA_ERR_DEVICE_BOUNDS
    close(got, reference(pool, q, want, tables, as_lens, 0.125), sel, 16, False, 6.0)


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_any_scale(scale):
    lens = [300, 20]
    pool, tables, q = make(lens, 8, 2, 128, torch.float16, 16, 2)
    run(pool, tables, q, lens, pick(lens, 2, 16, 9, 7), scale=scale)


def test_rising_scores_move_the_reference():
    lens = [2000]
    pool, tables, q = make(lens, 8, 1, 128, torch.bfloat16, 16)
    grow = torch.linspace(0.01, 3.0, 125, device=DEV)
    pool.k_cache[tables[0].long()] *= grow.view(-1, 1, 1, 1).to(torch.bfloat16)
    run(pool, tables, q, lens, pick(lens, 1, 16, 100, 8))


def test_the_largest_budget():
    lens = [4096 * 32, 77]
    pool, tables, q = make(lens, 4, 1, 64, torch.float16, 32, spare=0)
    run(pool, tables, q, lens, pick(lens, 1, 32, 4096, 9))
    assert pool.check() == pa.PA_OK


def test_captured_and_deterministic():
    lens = [900, 333, 64]
    pool, tables, q = make(lens, 16, 4, 128, torch.bfloat16, 16)
    sel, dl = pick(lens, 4, 16, 12, 10), i32(lens)
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pool.decode_selected(q, sel, tables, dl, 0.1, out=out)
    for i, ls in enumerate(([900, 333, 64], [899, 16, 1], [0, 333, 50])):
        dl.copy_(i32(ls))
        sel.copy_(pick(ls, 4, 16, 12, 20 + i))
        q.normal_()
        g.replay()
        close(out, reference(pool, q, sel, tables, ls, 0.1), sel, 16, False, 6.0)
        again = pool.decode_selected(q, sel, tables, dl, 0.1)
        assert torch.equal(again, out)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    again = pool.decode_selected(q, sel, tables, dl, 0.1, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(again, out)


def test_other_caches():
    lens = [100]
    pool, tables, q = make(lens, 8, 2, 64, torch.float16, 16)
    k, v = torch.randn_like(pool.k_cache), torch.randn_like(pool.v_cache)
    sel = pick(lens, 2, 16, 4, 11)
    got = pool.decode_selected(q, sel, tables, i32(lens), 0.125, k_cache=k, v_cache=v)
    close(got, reference(pool, q, sel, tables, lens, 0.125, k, v), sel, 16, False, 6.0)


def test_refusals():
    lens = [100, 90]
    pool, tables, q = make(lens, 8, 2, 64, torch.float16, 16)
    sel, dl, out = pick(lens, 2, 16, 4, 12), i32(lens), torch.full_like(q, 7.0)
    L = pa._sparse_lib()
    good = [pool.handle, q.data_ptr(), None, None, sel.data_ptr(), 4, tables.data_ptr(), tables.shape[1], dl.data_ptr(), 2, 8, 1,
            0.1, out.data_ptr(), None]
    for i, v in ((1, None), (4, None), (5, 0), (6, None), (7, 0), (8, None), (9, -1), (10, 0), (10, 7), (11, 0), (12, math.nan),
                 (12, math.inf), (13, None), (2, pool.k_cache.data_ptr()), (1, q.data_ptr() + 2), (13, out.data_ptr() + 8),
                 (13, q.data_ptr()), (13, q.data_ptr() + 64), (13, pool.v_cache.data_ptr()), (4, sel.data_ptr() + 2)):
        a = list(good)
        a[i] = v
        assert L.pa_decode_selected(*a) == pa.PA_ERR_INVALID_ARG, (i, v)
    for change in ({11: 9}, {10: 66}, {5: 4097}, {9: 2 ** 31 - 1}):
        a = list(good)
        for i, v in change.items():
            a[i] = v
        assert L.pa_decode_selected(*a) == pa.PA_ERR_UNSUPPORTED, change
    a = list(good)
    a[9] = 0
    assert L.pa_decode_selected(*a) == pa.PA_OK
    for kw in (dict(q=q.float()), dict(q=q[0]), dict(selected=sel[0]), dict(selected=sel.long()), dict(selected=sel[:, :1]),
               dict(out=out[:1]), dict(block_tables=tables[:1]), dict(context_lens=dl.long()), dict(k_cache=pool.k_cache),
               dict(k_cache=pool.k_cache.float(), v_cache=pool.v_cache.float()), dict(selected=sel[..., ::2])):
        with pytest.raises(ValueError):
            pool.decode_selected(**{**dict(q=q, selected=sel, block_tables=tables, context_lens=dl, scale=0.1), **kw})
    assert bool((out == 7.0).all()) and pool.check() == pa.PA_OK
