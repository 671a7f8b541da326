"""FP8 rows of rope_append: the codes themselves, and what the call leaves alone.

A code is the nearest E4M3 value to x / scale, scale the stored one. Values that are not rotated (v, and k's dimensions
from rot_dim on) are 16-bit: 448 x / max is a ratio of two small whole numbers there and meets a border between codes
exactly, again and again. But then x and scale are known, and the code is that of their fp32 quotient: equality.

The fp32 rotation is within |a| + |b| times 2^-20 of the 64-bit one and the quotient within 2^-24 of itself, so a
rotated value's code may differ from the one found in 64 bits only where x / scale lies that close to the border
between the two, and then by that one step. Rotated values come near a border by chance: with a probability of the
strip's width over a step.
"""
import random

import pytest
import torch

import test_gpu_rope_append as rope_test
from paged_kv_cache_223_gb300 import pagedattn as pa
from serving_reference import rotate

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def nearest_code(y):
    """The nearest E4M3 value to float64 y, ties to even, saturated; and the distance to the nearest border."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    z = (y / step).clamp(-448.0 / step, 448.0 / step)
    border = (z.abs() - torch.floor(z.abs()) - 0.5).abs() * step
    return (torch.round(z) * step).clamp(-448.0, 448.0), border


def parts(cache, pool):
    nb, hkv, bs, d = pool.geometry
    n = nb * hkv * bs
    return cache[:n * d].view(nb, hkv, bs, d), cache[n * d:].view(torch.float32).view(nb, hkv, bs)


@pytest.mark.parametrize("seed", range(401, 409))
def test_codes_and_other_rows(seed):
    rng = random.Random(seed)
    n, hkv, bs, inter = rng.choice([1, 2, 31, 150, 1300]), rng.choice([1, 2, 3, 8]), rng.choice([16, 32]), rng.random() < 0.5
    dt, rot = rng.choice([torch.bfloat16, torch.float16]), 16 * rng.randint(1, 8)
    pool, q, k, v, pos, slots = rope_test.make(seed, n, 4, hkv, 128, dt, bs, fp8=True, fused=rng.random() < 0.5)
    if n > 2:
        slots[1] = -1                                     # padding
    inv = rope_test.freqs(rot)
    pool.rope_append(q, k, v, pos, slots, pa.Rope(inv, interleaved=inter))
    assert pool.check() == pa.PA_OK
    live = slots >= 0
    blk, off = slots[live] // bs, slots[live] % bs
    unused = torch.ones(pool.geometry[0], bs, dtype=torch.bool, device=DEV)
    unused[blk, off] = False
    for cache, (x, mag) in ((pool.k_cache, rotate(k, pos, inv, inter)), (pool.v_cache, (v.double(), v.double() * 0))):
        codes, scales = parts(cache, pool)
        for t in (codes, scales.view(torch.int32)):       # whatever was not named keeps its words
            words = t.transpose(1, 2)[unused]
            assert bool((words == (0x7F if t is codes else 0x7F7F7F7F)).all())
        s = scales[blk, :, off].double()[..., None]
        got = codes[blk, :, off].view(torch.float8_e4m3fn).float().double()
        still = 128 if cache is pool.v_cache else 128 - rot   # dimensions that are not rotated
        y = x[live] / s
        plain = (x[live].float() / s.float()).double()        # one fp32 division
        assert torch.equal(got[..., 128 - still:], nearest_code(plain[..., 128 - still:])[0])
        y, got, mag = y[..., :128 - still], got[..., :128 - still], mag[live][..., :128 - still]
        want, border = nearest_code(y)
        wrong = got != want
        strip = mag / s * 2.0 ** -20 * 1.01 + y.abs() * 2.0 ** -23
        step = torch.exp2(torch.floor(torch.log2(torch.maximum(want.abs(), got.abs()).clamp(min=2.0 ** -6))) - 3)
        assert not bool((wrong & (border > strip)).any())
        assert not bool(((got - want).abs() > step).any())
        # the expected number of values in a strip, 16 times over (and a value or two)
        n_wrong, n_strip = int(wrong.sum()), float((2 * strip / step).clamp(max=1).sum())
        assert n_wrong <= 2 + 16 * n_strip, (n_wrong, n_strip)


def test_rows_too_small_for_a_scale():
    """A row whose largest value divided by 448 is no longer a number above 0 in fp32 is stored as zeros."""
    n, d = 6, 128
    pool = pa.Pool(1, 16, 1, d, torch.bfloat16, max_seqs=1, max_context_len=512, kv_format=pa.PA_KV_FP8_E4M3)
    k = torch.zeros(n, 1, d, dtype=torch.bfloat16, device=DEV)
    k.view(torch.int16)[:, :, 3:9] = 1                    # the smallest subnormal, 2^-133, among zeros
    slots = torch.arange(n, device=DEV)
    rope = pa.Rope(rope_test.freqs(d), scale=2.0 ** -12)
    pool.rope_append(None, k, k, torch.zeros(n, dtype=torch.int32, device=DEV), slots, rope)
    for cache, top in ((pool.k_cache, 2.0 ** -145), (pool.v_cache, 2.0 ** -133)):
        codes, scales = parts(cache, pool)
        value = codes[0, 0, :n].view(torch.float8_e4m3fn).float().double() * scales[0, 0, :n, None].double()
        x = torch.zeros(n, d, dtype=torch.float64, device=DEV)
        x[:, 3:9] = top
        assert bool(torch.isfinite(value).all()) and bool(((value - x).abs() <= top).all())
