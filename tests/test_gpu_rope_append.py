"""rope_append (pa_rope_append) against the rotation in 64 bits.

Tolerances: an output is rounded once to its type (half a step, eps / 2, relative; half the smallest
subnormal below that). Before it, the fp32 rotation: sine and cosine within 2 ulp (2^-22) of the angle
rounded to fp32 turns (pi 2^-24 radians), two products and a sum: (|a| + |b|) 2^-20 covers them. FP8 codes
are within half a step of E4M3 (2^-4 relative, 2^-10 scales in the subnormals).
"""
import numpy as np
import pytest
import torch

from paged_kv_cache_223_gb300 import pagedattn as pa
from serving_reference import rotate

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def make(seed, n, hq, hkv, d, dt, bs=16, fp8=False, fused=True, spare=20, maxpos=100000):
    g = torch.Generator(device=DEV).manual_seed(seed)
    qkv = torch.randn(n, (hq + 2 * hkv) * d, generator=g, device=DEV).to(dt)
    q, k, v = qkv.split([hq * d, hkv * d, hkv * d], 1)
    q, k, v = q.view(n, hq, d), k.view(n, hkv, d), v.view(n, hkv, d)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    nb = max(1, (n + spare + bs - 1) // bs)
    pos = torch.randint(0, maxpos, (n,), generator=g, device=DEV, dtype=torch.int32)
    slots = torch.randperm(nb * bs, generator=g, device=DEV)[:n].contiguous()
    pool = pa.Pool(nb, bs, hkv, d, dt, max_seqs=1, max_context_len=512,
                   kv_format=pa.PA_KV_FP8_E4M3 if fp8 else pa.PA_KV_16BIT)
    for c in (pool.k_cache, pool.v_cache):
        c.view(torch.uint8).fill_(0x7F)
    return pool, q, k, v, pos, slots


def close(got, ref, mag, what):
    dt = got.dtype
    tiny = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2
    tol = ref.abs() * torch.finfo(dt).eps / 2 + mag * 2.0 ** -20 * 1.01 + tiny
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), f"{what}: {int((err > tol).sum())} outside, worst {float((err - tol).max()):.3g}"


def rows_of(cache, slots, bs):
    return cache[slots // bs, :, slots % bs]


def check(pool, q, k, v, pos, slots, inv, inter, q_out, scale=1.0, k0=None, v0=None):
    bs = pool.geometry[2]
    ref, mag = rotate(q, pos, inv, inter, scale)
    close(q_out, ref, mag, "q")
    live = slots >= 0
    ref, mag = rotate(k, pos, inv, inter, scale)
    close(rows_of(pool.k_cache, slots[live], bs), ref[live], mag[live], "k")
    assert torch.equal(rows_of(pool.v_cache, slots[live], bs).view(torch.int16), v[live].contiguous().view(torch.int16))
    # nothing else was written
    used = torch.zeros(pool.geometry[0] * bs, dtype=torch.bool, device=DEV)
    used[slots[live]] = True
    rest = torch.arange(used.numel(), device=DEV)[~used]
    for c in (pool.k_cache, pool.v_cache):
        assert bool((rows_of(c, rest, bs).contiguous().view(torch.int16) == 0x7F7F).all())


def freqs(rot, base=500000.0):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


CASES = [
    # n, hq, hkv, d, dtype, bs, rot, interleaved, fused
    (1, 32, 8, 128, torch.bfloat16, 16, 128, False, True),
    (1, 1, 1, 64, torch.float16, 32, 16, True, False),
    (3, 5, 5, 64, torch.bfloat16, 16, 64, False, True),
    (7, 64, 8, 128, torch.float16, 16, 128, True, True),
    (33, 8, 1, 128, torch.bfloat16, 32, 64, False, False),
    (130, 12, 4, 64, torch.float16, 16, 32, False, True),
    (257, 20, 4, 128, torch.bfloat16, 16, 48, True, True),
    (1025, 64, 8, 128, torch.bfloat16, 16, 128, False, True),
    (2500, 16, 16, 64, torch.float16, 32, 64, True, False),
]


@pytest.mark.parametrize("case", CASES, ids=[f"n{c[0]}-h{c[1]}.{c[2]}-d{c[3]}-r{c[6]}{'i' if c[7] else 'h'}" for c in CASES])
def test_rotation_and_rows(case):
    n, hq, hkv, d, dt, bs, rot, inter, fused = case
    pool, q, k, v, pos, slots = make(n, n, hq, hkv, d, dt, bs, fused=fused)
    rope = pa.Rope(freqs(rot), interleaved=inter)
    out = pool.rope_append(q, k, v, pos, slots, rope)
    assert pool.check() == pa.PA_OK and out.is_contiguous()
    check(pool, q, k, v, pos, slots, freqs(rot), inter, out)


def test_far_and_negative_positions_and_scale():
    pool, q, k, v, pos, slots = make(5, 12, 8, 2, 128, torch.float16)
    pos = torch.tensor([0, 1, -1, 131071, 1 << 20, (1 << 24) + 1, 2 ** 31 - 1, -2 ** 31, 123456789, -77, 40000, 3],
                       dtype=torch.int32, device=DEV)
    inv = freqs(128, 10000.0)
    rope = pa.Rope(inv, scale=1.25)
    out = pool.rope_append(q, k, v, pos, slots, rope)
    check(pool, q, k, v, pos, slots, inv, False, out, scale=1.25)


def test_in_place_and_given_output_rows():
    for inter in (False, True):
        pool, q, k, v, pos, slots = make(8, 100, 8, 2, 128, torch.bfloat16, fused=True)
        rope = pa.Rope(freqs(128), interleaved=inter)
        q0 = q.clone()
        out = pool.rope_append(q, k, v, pos, slots, rope, q_out=q)
        assert out is q
        check(pool, q0, k, v, pos, slots, freqs(128), inter, q)
        wide = torch.full((100, 8 * 128 + 64), 7.0, dtype=torch.bfloat16, device=DEV)
        view = wide[:, :8 * 128].view(100, 8, 128)
        pool.rope_append(q0, k, v, pos, slots, rope, q_out=view)
        assert torch.equal(view, q) and bool((wide[:, 8 * 128:] == 7.0).all())


def test_padding_slots_and_keys_alone():
    pool, q, k, v, pos, slots = make(9, 50, 8, 2, 64, torch.float16)
    slots[::3] = -1
    rope = pa.Rope(freqs(64))
    out = pool.rope_append(q, k, v, pos, slots, rope)
    assert pool.check() == pa.PA_OK
    check(pool, q, k, v, pos, slots, freqs(64), False, out)
    for c in (pool.k_cache, pool.v_cache):
        c.view(torch.uint8).fill_(0x7F)
    assert pool.rope_append(None, k, v, pos, slots, rope) is None
    check(pool, q, k, v, pos, slots, freqs(64), False, out)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n", [1, 31, 700])
def test_fp8_pool(n, inter):
    hkv, bs, d = 4, 16, 128
    pool, q, k, v, pos, slots = make(n + 40, n, 8, hkv, d, torch.bfloat16, bs, fp8=True)
    k[0] = 0.0                                   # an all-zero row: scale 1
    rope = pa.Rope(freqs(64), interleaved=inter)
    out = pool.rope_append(q, k, v, pos, slots, rope)
    assert pool.check() == pa.PA_OK
    ref, mag = rotate(q, pos, freqs(64), inter)
    close(out, ref, mag, "q")
    nb = pool.geometry[0]
    for cache, x in ((pool.k_cache, rotate(k, pos, freqs(64), inter)[0]), (pool.v_cache, v.double())):
        codes = cache[:nb * hkv * bs * d].view(torch.float8_e4m3fn).float().double().view(nb, hkv, bs, d)
        scales = cache[nb * hkv * bs * d:].view(torch.float32).double().view(nb, hkv, bs)
        c, s = codes[slots // bs, :, slots % bs], scales[slots // bs, :, slots % bs]
        amax = x.abs().amax(-1)
        want = torch.where(amax > 0, amax / 448, 1.0)
        assert bool(((s - want).abs() <= want * 2.0 ** -19).all())
        tol = x.abs() * 2.0 ** -4 + want[..., None] * (2.0 ** -10 + 448 * 2.0 ** -18)
        assert bool(((c * s[..., None] - x).abs() <= tol).all())
        # nearest codes: the error is at most half a step almost everywhere, a step only on a border
        assert float(codes.abs()[torch.isfinite(codes)].max()) <= 448


def test_fp8_unrotated_rows_equal_cache_write():
    """At position 0 the fused append stores what pa_cache_write stores for the same rows, bit for bit."""
    for fp8 in (False, True):
        pool, q, k, v, pos, slots = make(60, 77, 8, 2, 128, torch.float16, fp8=fp8)
        pos.zero_()
        pool.rope_append(q, k, v, pos, slots, pa.Rope(freqs(128)))
        a = (pool.k_cache.clone(), pool.v_cache.clone())
        pool.cache_write(k.contiguous(), v.contiguous(), slots)
        assert torch.equal(a[0].view(torch.uint8), pool.k_cache.view(torch.uint8))
        assert torch.equal(a[1].view(torch.uint8), pool.v_cache.view(torch.uint8))


def test_slots_outside_the_pool_are_skipped_and_flagged():
    pool, q, k, v, pos, slots = make(61, 9, 4, 2, 64, torch.bfloat16)
    good = slots.clone()
    slots[4] = pool.geometry[0] * pool.geometry[2]
    good[4] = -1
    rope = pa.Rope(freqs(64))
    out = pool.rope_append(q, k, v, pos, slots, rope)
    assert pool.check() == pa.PA_ERR_DEVICE_BOUNDS
    check(pool, q, k, v, pos, good, freqs(64), False, out)


def test_refusals_on_the_host():
    pool, q, k, v, pos, slots = make(62, 9, 4, 2, 64, torch.bfloat16, fused=False)
    rope = pa.Rope(freqs(64))
    for bad in (lambda: pool.rope_append(q[:, :, :32], k, v, pos, slots, rope),
                lambda: pool.rope_append(q, k[:8], v, pos, slots, rope),
                lambda: pool.rope_append(q, k, v, pos.long(), slots, rope),
                lambda: pool.rope_append(q, k, v, pos, slots.int(), rope),
                lambda: pool.rope_append(q.half(), k, v, pos, slots, rope),
                lambda: pool.rope_append(q, k, v, pos, slots, rope, q_out=q[:8]),
                lambda: pool.rope_append(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, pos, slots, rope),
                lambda: pool.rope_append(q, k[:1].expand(9, 2, 64), v, pos, slots, rope),
                lambda: pool.rope_append(q.cpu(), k, v, pos, slots, rope)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(pa.PagedAttnError):       # more rotated dimensions than the pool's heads have
        pool.rope_append(q, k, v, pos, slots, pa.Rope(freqs(128)))
    buf = torch.empty(9 * 4 * 64 + 1, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(pa.PagedAttnError):       # rows that do not start on 16 bytes
        pool.rope_append(buf[1:].view(9, 4, 64), k, v, pos, slots, rope)
    rows = torch.zeros(10, 12, 64, dtype=torch.bfloat16, device=DEV)          # q | k | v | room for an output
    q, k, v, room = rows[:9, :4], rows[:9, 4:6], rows[:9, 6:8], rows[:9, 8:]
    for over in (rows[:9, 1:5], rows[:9, 3:7], rows[:9, 7:11], rows[1:, :4], rows.view(-1)[:9 * 4 * 64].view(9, 4, 64)):
        with pytest.raises(pa.PagedAttnError):   # an output over other rows of q, or of k or v
            pool.rope_append(q, k, v, pos, slots, rope, q_out=over)
    assert pool.rope_append(q, k, v, pos, slots, rope, q_out=room) is room
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    out = pool.rope_append(e, e[:, :2], e[:, :2], pos[:0], slots[:0], rope)
    assert out.shape == (0, 4, 64)


def test_other_stream_and_graph():
    pool, q, k, v, pos, slots = make(63, 200, 8, 2, 128, torch.bfloat16)
    rope = pa.Rope(freqs(128))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = pool.rope_append(q, k, v, pos, slots, rope, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    check(pool, q, k, v, pos, slots, freqs(128), False, out)
    q_out = torch.empty_like(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pool.rope_append(q, k, v, pos, slots, rope, q_out=q_out)
    q.mul_(2.0)
    pos.add_(5)
    g.replay()
    check(pool, q, k, v, pos, slots, freqs(128), False, q_out)
