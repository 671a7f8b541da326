"""select_blocks (pa_select_blocks) against its definition. Scores are sums of whole numbers times powers of two, so they
are exact in fp32 as in 64 bits, and the lists are equal."""
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_223_gb300 import pagedattn as pa
from sparse_reference import ceil_div, select

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def make(lens, hq, hkv, d, dt, bs, q_len=1, seed=0, spare=2, levels=127, stride=None):
    """A pool, tables, bounds of random codes (hi >= lo) with steps of a few sizes, and q."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    blocks = [ceil_div(n, bs) for n in lens]
    nb = sum(blocks) + spare
    pool = pa.Pool(nb, bs, hkv, d, dt, max_seqs=1, max_q_heads=hq, max_context_len=512)
    codes = torch.randint(-levels, levels + 1, (nb, hkv, 2, d), generator=g, device=DEV).sort(2, descending=True).values
    steps = torch.exp2(torch.randint(-7, -4, (nb, hkv), generator=g, device=DEV).float())
    ids = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    stride = stride or max([1] + blocks)
    tables, at = torch.full((len(lens), stride), -1, dtype=torch.int32, device=DEV), 0
    for i, k in enumerate(blocks):
        tables[i, :k] = ids[at:at + k]
        at += k
    q = torch.randn(len(lens), q_len, hq, d, generator=g, device=DEV).to(dt)
    return pool, codes, steps, tables, q


def buffer(codes, steps):
    return torch.cat([codes.to(torch.int8).view(-1).view(torch.uint8), steps.view(-1).view(torch.uint8)])


def expected(q, codes, steps, tables, lens, bs, budget, first, last):
    B, _, hq, d = q.shape
    hkv = codes.shape[1]
    c, s, t, x = (v.cpu().numpy() for v in (codes, steps.double(), tables, q.double()))
    return np.stack([np.stack([select(x[b][:, h * (hq // hkv):(h + 1) * (hq // hkv)].reshape(-1, d), c[:, h], s[:, h],
                                      t[b], lens[b], bs, budget, first, last) for h in range(hkv)]) for b in range(B)])


def run(pool, codes, steps, tables, q, lens, budget, first=1, last=2, **kw):
    got = pool.select_blocks(q, buffer(codes, steps), tables, i32(lens), budget, first, last, **kw)
    want = expected(q, codes, steps, tables, lens, pool.geometry[2], budget, first, last)
    assert np.array_equal(got.cpu().numpy(), want)
    return want


@pytest.mark.parametrize("lens,hq,hkv,d,dt,bs,q_len,budget,first,last", [
    ([1], 1, 1, 64, torch.float16, 16, 1, 1, 0, 1),
    ([1000], 8, 8, 128, torch.bfloat16, 16, 1, 7, 1, 2),
    ([333, 16, 17, 5000], 32, 8, 128, torch.bfloat16, 16, 1, 20, 1, 4),
    ([4097, 900], 16, 4, 64, torch.float16, 32, 4, 33, 2, 2),          # 16 rows
    ([3000, 77, 8], 12, 4, 128, torch.float16, 16, 8, 16, 0, 3),       # 24 rows
    ([2100, 2099], 64, 2, 64, torch.bfloat16, 16, 1, 64, 3, 5),        # a group of 32
    ([999, 1500, 64], 20, 4, 128, torch.bfloat16, 32, 5, 12, 1, 2),    # 25 rows
    ([20000], 8, 1, 128, torch.float16, 16, 1, 128, 1, 2),
    ([70000, 40, 33000], 4, 2, 64, torch.bfloat16, 16, 2, 300, 4, 4),
    ([100], 4, 2, 64, torch.float16, 16, 1, 4096, 1, 2),
    ([131072 + 5], 16, 2, 128, torch.bfloat16, 16, 1, 4096, 1, 2),
    ([700] * 70, 16, 16, 64, torch.float16, 16, 1, 9, 1, 2),
])
def test_selection(lens, hq, hkv, d, dt, bs, q_len, budget, first, last):
    pool, codes, steps, tables, q = make(lens, hq, hkv, d, dt, bs, q_len, seed=budget)
    run(pool, codes, steps, tables, q, lens, budget, first, last)
    assert pool.check() == pa.PA_OK


@pytest.mark.parametrize("kind", ["all equal", "few levels", "zeros", "one bit"])
def test_ties_go_to_the_lowest_index(kind):
    lens = [5000, 1700]
    pool, codes, steps, tables, q = make(lens, 8, 2, 64, torch.float16, 16, seed=3, levels=1)
    steps.fill_(0.25)
    if kind == "all equal":
        codes[:] = codes[:1]
    elif kind == "zeros":
        codes.zero_(), steps.zero_()
    elif kind == "one bit":                              # two scores only
        q[:] = 0
        q[..., 5] = 1.0
        codes[:, :, 1] = codes[:, :, 0]
        codes[:, :, :, 5] = (torch.arange(codes.shape[0], device=DEV) % 3 == 1).view(-1, 1, 1).long()
    for budget in (3, 4, 60, 105, 106, 107, 300):
        run(pool, codes, steps, tables, q, lens, budget, 1, 2)
    assert pool.check() == pa.PA_OK


def test_the_largest_sums():
    """Codes of +-127 everywhere: sums of 128 and 64 products at the ends of their range, alternating by one."""
    for d in (64, 128):
        lens = [4000]
        pool, codes, steps, tables, q = make(lens, 8, 1, d, torch.float16, 16, seed=4)
        q[:] = 127.0 * torch.where(torch.arange(d, device=DEV) % 2 == 0, 1.0, -1.0)
        codes[:, :, 0], codes[:, :, 1] = 127, -127
        at = torch.arange(codes.shape[0], device=DEV)
        codes[at, 0, 0, 2 * (at % 8)] -= (at % 5)
        steps.fill_(1.0)
        run(pool, codes, steps, tables, q, lens, 40)
        q[:, :, :4] *= -1
        codes[:, :, 0], codes[:, :, 1] = -127, -127       # negative scores
        codes[at, 0, 0, 2 * (at % 8)] += (at % 5)
        run(pool, codes, steps, tables, q, lens, 41)


def test_steps_far_apart():
    lens = [9000]
    pool, codes, steps, tables, q = make(lens, 4, 2, 128, torch.bfloat16, 16, seed=5)
    steps.copy_(torch.exp2(torch.randint(-60, 60, steps.shape, device=DEV).float()))
    q *= torch.exp2(torch.tensor([-30.0, 0.0, 25.0, 3.0], device=DEV)).view(1, 1, 4, 1)
    run(pool, codes, steps, tables, q, lens, 50)


@pytest.mark.parametrize("q_len", [1, 3])
def test_no_numbers(q_len):
    lens = [3000, 2000, 2500]
    pool, codes, steps, tables, q = make(lens, 8, 2, 64, torch.bfloat16, 16, q_len, seed=6)
    steps[tables[0, 90].long(), 0] = math.inf             # a block that holds no numbers is wanted
    codes[tables[0, 90].long(), 0] = 0
    q[0, 0, 1, 5] = math.nan                              # a row that does not count
    q[1, :, :4] = math.inf                                # a group without a row that counts: the first blocks
    q[2, 0] = 0.0
    got = run(pool, codes, steps, tables, q, lens, 11)
    assert 90 in got[0, 0] and got[1, 0].tolist() == list(range(9)) + [123, 124]
    assert pool.check() == pa.PA_OK


def test_padding_and_short_contexts():
    lens = [0, 3, 800, 0, 161]
    pool, codes, steps, tables, q = make(lens, 8, 2, 128, torch.float16, 16, 3, seed=7, stride=60)
    got = run(pool, codes, steps, tables, q, lens, 10, 1, 2)
    assert (got[0] == -1).all() and (got[3] == -1).all()
    assert pool.check() == pa.PA_OK


@pytest.mark.parametrize("what", ["negative", "long", "shorter than the rows"])
def test_lengths_that_do_not_fit(what):
    lens = [900, 800]
    pool, codes, steps, tables, q = make(lens, 8, 2, 64, torch.float16, 16, 4, seed=8)
    bad, as_if = {"negative": (-5, 0), "long": (57 * 16 + 1, 57 * 16), "shorter than the rows": (3, 3)}[what]
    tables[1] = tables[0]
    got = pool.select_blocks(q, buffer(codes, steps), tables, i32([900, bad]), 12).cpu().numpy()
    assert pool.check() == pa.PA_ERR_DEVICE_BOUNDS
    assert np.array_equal(got, expected(q, codes, steps, tables, [900, as_if], 16, 12, 1, 2))


def test_ids_outside_the_pool_score_lowest():
    lens = [900]
    pool, codes, steps, tables, q = make(lens, 8, 2, 64, torch.float16, 16, seed=9)
    want = expected(q, codes, steps, tables, lens, 16, 20, 1, 2)
    gone = [int(i) for i in want[0, 0][3:6]]
    bad = tables.clone()
    bad[0, gone[0]], bad[0, gone[1]], bad[0, gone[2]] = -1, pool.geometry[0], 2 ** 31 - 1
    got = pool.select_blocks(q, buffer(codes, steps), bad, i32(lens), 20).cpu().numpy()
    assert pool.check() == pa.PA_ERR_DEVICE_BOUNDS
    assert np.array_equal(got, expected(q, codes, steps, bad, lens, 16, 20, 1, 2)) and not set(gone) & set(got[0, 0].tolist())


def test_the_longest_tables():
    """PA_SELECT_MAX_BLOCKS entries, all naming the same few blocks: ties everywhere."""
    n, bs = 262144, 32
    pool, codes, steps, tables, q = make([bs * 40], 4, 1, 64, torch.float16, bs, seed=10)
    tables = (torch.arange(n, dtype=torch.int32, device=DEV) % 40).view(1, n)
    got = run(pool, codes, steps, tables, q, [n * bs], 4096)
    assert pool.check() == pa.PA_OK and len(set(got[0, 0].tolist())) == 4096
    with pytest.raises(pa.PagedAttnError) as e:
        pool.select_blocks(q, buffer(codes, steps), torch.zeros(1, n + 1, dtype=torch.int32, device=DEV), i32([5]), 8)
    assert e.value.status == pa.PA_ERR_UNSUPPORTED


def test_captured_and_on_streams():
    lens = [3000, 400]
    pool, codes, steps, tables, q = make(lens, 8, 2, 128, torch.bfloat16, 16, seed=11)
    dl, buf = i32(lens), buffer(codes, steps)
    out = torch.zeros(2, 2, 16, dtype=torch.int32, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pool.select_blocks(q, buf, tables, dl, 16, out=out)
    for ls in ([3000, 400], [100, 399], [0, 256], [2999, 257]):
        dl.copy_(i32(ls))
        q.normal_()
        g.replay()
        assert np.array_equal(out.cpu().numpy(), expected(q, codes, steps, tables, ls, 16, 16, 1, 2))
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    x = pool.select_blocks(q, buf, tables, dl, 16, stream=a)
    y = pool.select_blocks(q, buf, tables, dl, 30, stream=b)
    torch.cuda.synchronize()
    assert torch.equal(x, out)
    assert np.array_equal(y.cpu().numpy(), expected(q, codes, steps, tables, [2999, 257], 16, 30, 1, 2))


def test_refusals():
    lens = [900, 800]
    pool, codes, steps, tables, q = make(lens, 8, 2, 64, torch.float16, 16, seed=12)
    L, buf, dl = pa._sparse_lib(), buffer(codes, steps), i32(lens)
    out = torch.full((2, 2, 8), 5, dtype=torch.int32, device=DEV)
    good = [pool.handle, q.data_ptr(), buf.data_ptr(), tables.data_ptr(), tables.shape[1], dl.data_ptr(), 2, 8, 1, 8, 1, 2,
            out.data_ptr(), None]
    for i, v in ((1, None), (2, None), (3, None), (4, 0), (5, None), (6, -1), (7, 0), (7, 9), (8, 0), (9, 0), (9, 2), (10, -1),
                 (10, 7), (11, 0), (11, 8), (12, None), (1, q.data_ptr() + 2), (2, buf.data_ptr() + 1), (12, out.data_ptr() + 2),
                 (12, q.data_ptr()), (12, tables.data_ptr() + 4), (12, buf.data_ptr() + 16), (12, dl.data_ptr())):
        a = list(good)
        a[i] = v
        assert L.pa_select_blocks(*a) == pa.PA_ERR_INVALID_ARG, (i, v)
    for change in ({8: 9}, {7: 66}, {9: 4097}, {8: 2 ** 31 - 1}, {6: 2 ** 31 - 1}):
        a = list(good)
        for i, v in change.items():
            a[i] = v
        assert L.pa_select_blocks(*a) == pa.PA_ERR_UNSUPPORTED, change
    a = list(good)
    a[8], a[11] = 2, 1                                    # two rows may lie in two blocks
    assert L.pa_select_blocks(*a) == pa.PA_ERR_INVALID_ARG
    a = list(good)
    a[6] = 0
    assert L.pa_select_blocks(*a) == pa.PA_OK
    for kw in (dict(q=q.float()), dict(q=q[0]), dict(q=q.transpose(0, 2)), dict(bounds=buf[1:]), dict(out=out[:1]),
               dict(out=out.long()), dict(block_tables=tables[:1]), dict(context_lens=dl[:1]), dict(budget=7, out=out)):
        with pytest.raises(ValueError):
            pool.select_blocks(**{**dict(q=q, bounds=buf, block_tables=tables, context_lens=dl, budget=8), **kw})
    assert bool((out == 5).all()) and pool.check() == pa.PA_OK
