"""prefill_packed at the ends of what its plan can hold."""
import math

import pytest
import torch

from paged_kv_cache_223_gb300 import pagedattn as pa
from serving_reference import packed_attention
from test_gpu_packed import close

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def test_a_decreasing_cu_q_is_flagged_and_bounded():
    """2048 sequences, every other one naming all rows: flagged, and not 1024 times a call's work."""
    T, n, hq, hkv, d, bs = 4096, 2048, 64, 8, 128, 16
    g = torch.Generator(device=DEV).manual_seed(71)
    pool = pa.Pool(T // bs, bs, hkv, d, torch.bfloat16, max_seqs=1, max_context_len=512)
    pool.k_cache.normal_(generator=g), pool.v_cache.normal_(generator=g)
    q = torch.randn(T + 3, hq, d, generator=g, device=DEV).to(torch.bfloat16)
    tables = torch.arange(T // bs, dtype=torch.int32, device=DEV).repeat(n, 1)
    lens, whole, wrong = i32([T] * n), i32([0, T]), i32([0, T] * (n // 2) + [0])
    out = torch.full_like(q, 7.0)

    def timed(cu):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        pool.prefill_packed(q, cu, tables, lens, 1 / math.sqrt(d), out=out)
        b.record()
        b.synchronize()
        return a.elapsed_time(b)

    timed(whole)
    one = min(timed(whole) for _ in range(3))
    assert pool.check() == pa.PA_OK
    ref = out.clone()
    out.fill_(7.0)
    many = timed(wrong)
    assert pool.check() == pa.PA_ERR_DEVICE_BOUNDS
    assert many < 100 * one, (many, one)
    assert bool((out[T:] == 7.0).all())               # rows of no sequence
    timed(whole)
    assert pool.check() == pa.PA_OK and torch.equal(out, ref)


def test_the_longest_context():
    """PA_PACKED_MAX_CONTEXT tokens, of blocks whose keys are 0 and values 1: weights of 1 and sums of whole numbers,
    so the output is 1. One block more is flagged, and the sequence beside it keeps its result."""
    most, hq, d, bs, shared = 1 << 29, 2, 64, 32, 8192
    pool = pa.Pool(shared + 2, bs, 1, d, torch.float16, max_seqs=1, max_q_heads=hq, max_context_len=512)
    g = torch.Generator(device=DEV).manual_seed(72)
    pool.k_cache.normal_(generator=g), pool.v_cache.normal_(generator=g)
    pool.k_cache[:shared] = 0.0
    pool.v_cache[:shared] = 1.0
    tables = (torch.arange(most // bs + 1, dtype=torch.int32, device=DEV) % shared).repeat(2, 1)
    tables[1, 0], tables[1, 1] = shared + 1, shared
    q = torch.randn(1 + 40, hq, d, generator=g, device=DEV).half()
    cu = i32([0, 1, 41])
    out = pool.prefill_packed(q, cu, tables, i32([most, 50]), 0.125)
    assert pool.check() == pa.PA_OK
    assert bool((out[0] == 1.0).all())
    ref, mag = packed_attention(q[1:], pool.k_cache, pool.v_cache, [0, 40], tables[1:], [50], 0.125)
    close(out[1:], ref, mag)
    long = pool.prefill_packed(q, cu, tables, i32([most + bs, 50]), 0.125)
    assert pool.check() == pa.PA_ERR_DEVICE_BOUNDS and torch.equal(long[1:], out[1:])


def test_a_long_context_that_is_not_cut():
    """2^28 tokens of one row beside rows that fill the GPU: one block works through them for about three seconds while
    its next unit waits."""
    long, rest, hq, d, bs, shared = 1 << 28, 640, 128, 64, 32, 8192
    pool = pa.Pool(shared, bs, 1, d, torch.float16, max_seqs=1, max_q_heads=hq, max_context_len=512)
    pool.k_cache.zero_(), pool.v_cache.fill_(1.0)
    tables = (torch.arange(long // bs, dtype=torch.int32, device=DEV) % shared).repeat(2, 1)
    q = torch.ones(1 + rest, hq, d, dtype=torch.float16, device=DEV)
    out = pool.prefill_packed(q, i32([0, 1, 1 + rest]), tables, i32([long, rest]), 0.125)
    assert pool.check() == pa.PA_OK
    assert bool((out[1:] == 1.0).all())


@pytest.mark.parametrize("scores", ["flat", "random", "rising", "falling"])
@pytest.mark.parametrize("log2,d,dt", [(15, 64, torch.float16), (18, 128, torch.bfloat16), (20, 64, torch.float16),
                                       (20, 128, torch.float16)])
def test_sums_over_long_contexts_that_are_not_cut(log2, d, dt, scores):
    """One row behind 2^log2 tokens beside rows that fill the GPU, values between 1 and 2. The tolerance of the packed
    prompts' tests, and what an accumulator drops of the products added to it: 2^-26 of the sum each, for the 128
    tiles of 128 keys that it takes, 2^-12 in all."""
    long, rest, hq, bs = 1 << log2, 9800, 8, 32
    g = torch.Generator(device=DEV).manual_seed(73)
    nb = long // bs
    pool = pa.Pool(nb, bs, 1, d, dt, max_seqs=1, max_q_heads=hq, max_context_len=512)
    pool.k_cache.normal_(generator=g), pool.v_cache.uniform_(1.0, 2.0, generator=g)
    q = torch.randn(1 + rest, hq, d, generator=g, device=DEV).to(dt)
    scale = 1 / math.sqrt(d)
    if scores == "flat":
        q.zero_()
    elif scores != "random":                          # from 0 to 24 along the context, or back
        q[0] = 0.0
        q[0, :, 0] = 4.0
        ramp = torch.linspace(0.0, 6.0 / scale, long, device=DEV)
        pool.k_cache.view(long, d)[:, 0] = (ramp if scores == "rising" else ramp.flip(0)).to(dt)
    tables = torch.arange(nb, dtype=torch.int32, device=DEV).repeat(2, 1)
    out = pool.prefill_packed(q, i32([0, 1, 1 + rest]), tables, i32([long, rest]), scale)
    assert pool.check() == pa.PA_OK
    K, V = pool.k_cache.view(long, d), pool.v_cache.view(long, d)
    s = torch.cat([q[0].double() @ k.double().T for k in K.split(1 << 18)], 1) * scale
    w = torch.softmax(s, 1)
    ref = sum(x @ v.double() for x, v in zip(w.split(1 << 18, 1), V.split(1 << 18)))      # all values > 0: sum p|v| too
    h = torch.finfo(dt).eps / 2
    err = (out[0].double() - ref).abs()
    assert bool((err <= ref * (2.01 * h + 2.0 ** -12 + 2.0 ** -12)).all()), float((err / ref).max())
