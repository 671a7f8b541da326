"""rope_append, prefill_packed, adjust_logits and token_probs at seeded random sizes, against their 64-bit definitions."""
import math
import random

import pytest
import torch

import test_gpu_logits as logits_test
import test_gpu_packed as packed_test
import test_gpu_rope_append as rope_test
from paged_kv_cache_223_gb300 import pagedattn as pa

pytestmark = pytest.mark.gpu
HALVES = [torch.bfloat16, torch.float16]


def size(rng, lo, hi):
    """Even over the magnitudes from lo to hi."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


@pytest.mark.parametrize("seed", range(101, 125))
def test_packed(seed):
    rng = random.Random(seed)
    d, hkv, bs = rng.choice([64, 128]), rng.choice([1, 2, 3, 4, 8]), rng.choice([16, 32])
    group = rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 12, 16, 33, 64, 128) if g * hkv <= 128])
    n = rng.choice([1, 1, 2, 3, 5, 9, 40])
    longest = max(1, min(2500, 300000 // (group * hkv * n)))
    new = [rng.choice([0, 1, size(rng, 1, longest), size(rng, 1, longest)]) for _ in range(n)]
    old = [rng.choice([0, 0, size(rng, 1, 200), size(rng, 1, 20000 if n < 6 else 1000)]) for _ in range(n)]
    packed_test.check(*packed_test.make(seed, new, old, group * hkv, hkv, d, rng.choice(HALVES), bs,
                                        spare_rows=rng.choice([0, 5]), first=rng.choice([0, 3])))


@pytest.mark.parametrize("seed", range(201, 217))
def test_rope(seed):
    rng = random.Random(seed)
    d, n, hkv, hq = rng.choice([64, 128]), size(rng, 1, 4000), rng.choice([1, 2, 3, 5, 8]), rng.choice([1, 2, 7, 16, 64])
    inv, inter = rope_test.freqs(16 * rng.randint(1, d // 16)), rng.random() < 0.5
    pool, q, k, v, pos, slots = rope_test.make(seed, n, hq, hkv, d, rng.choice(HALVES), rng.choice([16, 32]),
                                               fused=rng.random() < 0.5)
    out = pool.rope_append(q, k, v, pos, slots, pa.Rope(inv, interleaved=inter))
    rope_test.check(pool, q, k, v, pos, slots, inv, inter, out)


@pytest.mark.parametrize("seed", range(301, 333))
def test_logits(seed):
    rng = random.Random(seed)
    V, rows = size(rng, 1, 393216), rng.choice([1, 1, 2, 3, 6, 9])
    B = max(1, min(size(rng, 1, 400), 10_000_000 // (V * rows)))
    S, biases = rng.choice([0, 1, 40, 600, 5000, 20000]), rng.choice([0, 1, 30, 2000])
    if B > 64:
        S, biases = min(S, 600), min(biases, 30)
    x, kw, t = logits_test.make(seed, B, rows, V, rng.choice(HALVES + [torch.float32]), S, biases, rng.random() < 0.5,
                                rng.random() < 0.7, rng.choice([0, 0, 1, 3, 4, 8]))
    ref, mag = logits_test.adjusted(x, **kw)
    logits_test.close_adjusted(pa.adjust_logits(x, **kw), ref, mag)
    logits_test.close_probs(pa.token_probs(x, t, **kw), logits_test.probs(ref, t), mag, t)
