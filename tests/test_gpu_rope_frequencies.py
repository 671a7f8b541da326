"""Angles of rope_append at far positions: frequencies of either sign, to 2^-64 turns per position.

Near a whole number of turns the sine is small, so its relative rounding leaves the angle itself to be seen:
with a = 1 and b = 0 the pair's second element is scale sin(angle). Tolerance: the frequency is a whole number of
2^-64 turns (p 2^-64 turns at position p); the reduced angle's rounding to fp32 and the sine's 2 ulp, 2^-21 relative;
the output's rounding, 2^-11.
"""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from paged_kv_cache_223_gb300 import pagedattn as pa

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def arctan_inverse(n, bits):
    """arctan(1 / n) 2^bits, by its series in whole numbers."""
    total, term, k = 0, (1 << bits) // n, 0
    while term:
        total += term // (2 * k + 1) * (-1 if k & 1 else 1)
        term //= n * n
        k += 1
    return total


TWO_PI = Fraction(8 * (4 * arctan_inverse(5, 300) - arctan_inverse(239, 300)), 1 << 300)   # Machin's formula


def rows(n, h, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(n, h, 128, generator=g, device=DEV).half()


def append(pool, q, pos, rope):
    n = q.shape[0]
    kv = q[:, :1].contiguous()
    return pool.rope_append(q, kv, kv, pos, torch.full((n,), -1, dtype=torch.int64, device=DEV), rope)


def test_a_negative_frequency_is_a_negative_position():
    """p (-f) and (-p) f are one angle: equal bit for bit."""
    n = 4000
    pool = pa.Pool(1, 16, 1, 128, torch.float16, max_seqs=1, max_context_len=512)
    q = rows(n, 4, 1)
    pos = torch.arange(2 ** 31 - 1 - n, 2 ** 31 - 1, device=DEV).to(torch.int32)
    f = [10000.0 ** (-2.0 * i / 128) * (1 + i % 3 * 0.37) for i in range(64)]
    for inter in (False, True):
        a = append(pool, q, pos, pa.Rope([-x for x in f], interleaved=inter))
        b = append(pool, q, -pos, pa.Rope(f, interleaved=inter))
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_angles_near_whole_turns(sign):
    freqs = [sign * w for w in (0.3, 1.0, 1e-4, 123.456, 7.5e-3, 1e6, 2.0 ** -30, 0.05)]
    scale = 1024.0
    pool = pa.Pool(1, 16, 1, 128, torch.float16, max_seqs=1, max_context_len=512)
    rope = pa.Rope(freqs, scale=scale)
    pos, want = [], []
    for w in freqs:
        turns = Fraction(w) / TWO_PI
        unit = round(turns * 2 ** 64) % 2 ** 64
        p = np.arange(2 ** 31 - 400000, 2 ** 31, dtype=np.uint64)
        with np.errstate(over="ignore"):
            off = (p * np.uint64(unit)).view(np.int64)            # 2^-64 turns from a whole number of them
        p = int(p[np.abs(off.astype(np.float64)).argmin()])
        rest = turns * p - round(turns * p)
        pos.append(p)
        want.append(scale * math.sin(float(rest * TWO_PI)))
    q = torch.zeros(len(freqs), 1, 128, dtype=torch.float16, device=DEV)
    q[:, :, :len(freqs)] = 1.0
    out = append(pool, q, torch.tensor(pos, dtype=torch.int32, device=DEV), rope)
    for i, (p, s) in enumerate(zip(pos, want)):
        got = float(out[i, 0, len(freqs) + i])
        tol = abs(s) * (2.0 ** -11 + 2.0 ** -21) + scale * p * 2.0 ** -64 * 2 * math.pi + 2.0 ** -25
        assert abs(got - s) <= tol, (freqs[i], p, got, s, tol)


def test_frequencies_of_a_base():
    pool = pa.Pool(1, 16, 1, 128, torch.float16, max_seqs=1, max_context_len=512)
    q = rows(100, 2, 2)
    pos = torch.arange(100, dtype=torch.int32, device=DEV) * 77
    for rot, base in ((128, 10000.0), (64, 500000.0)):
        a = append(pool, q, pos, pa.Rope.from_base(rot, base, interleaved=True, scale=0.5))
        b = append(pool, q, pos, pa.Rope([base ** (-2.0 * i / rot) for i in range(rot // 2)], True, 0.5))
        assert torch.equal(a, b)
