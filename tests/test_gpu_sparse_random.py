"""The sparse decode step's calls at seeded random sizes: heads, groups, rows, lengths, budgets, block sizes, formats."""
import random

import numpy as np
import pytest
import torch

from paged_kv_cache_223_gb300 import pagedattn as pa
import test_gpu_decode_selected as A
import test_gpu_key_bounds as K
import test_gpu_select_blocks as S

pytestmark = pytest.mark.gpu


def shape(rng):
    d = rng.choice([64, 128])
    while True:
        hkv, G, q_len = rng.choice([1, 2, 3, 8]), rng.choice([1, 2, 3, 4, 5, 8, 16, 32]), rng.choice([1, 1, 2, 3, 5, 8, 17, 32])
        if G * q_len <= 32:
            break
    b = rng.choice([1, 2, 5, 20])
    most = rng.choice([20, 300, 3000])
    lens = [rng.choice([0, 1, rng.randint(1, most), most]) for _ in range(b)]
    lens = [n if n == 0 or n >= q_len else q_len for n in lens]
    return dict(d=d, hkv=hkv, hq=hkv * G, q_len=q_len, bs=rng.choice([16, 32]), lens=lens,
                dt=rng.choice([torch.float16, torch.bfloat16]), fp8=d == 128 and rng.random() < 0.4)


@pytest.mark.parametrize("seed", range(24))
def test_selection(seed):
    rng = random.Random(seed)
    c = shape(rng)
    last = rng.randint(-(-(c["q_len"] - 1) // c["bs"]) + 1, 6)
    first = rng.choice([0, 1, 3])
    budget = first + last + rng.choice([0, 1, 5, 30, 90])
    pool, codes, steps, tables, q = S.make(c["lens"], c["hq"], c["hkv"], c["d"], c["dt"], c["bs"], c["q_len"], seed=seed,
                                           levels=rng.choice([1, 10, 127]), stride=rng.choice([None, 250]))
    S.run(pool, codes, steps, tables, q, c["lens"], budget, first, last)
    assert pool.check() == pa.PA_OK


@pytest.mark.parametrize("seed", range(24))
def test_attention(seed):
    rng = random.Random(100 + seed)
    c = shape(rng)
    pool, tables, q = A.make(c["lens"], c["hq"], c["hkv"], c["d"], c["dt"], c["bs"], c["q_len"], c["fp8"], seed=seed)
    sel = A.pick(c["lens"], c["hkv"], c["bs"], rng.choice([1, 2, 7, 40]), seed, rng.choice(["ascending", "any", "holes"]))
    A.run(pool, tables, q, c["lens"], sel)
    assert pool.check() == pa.PA_OK


@pytest.mark.parametrize("seed", range(16))
def test_bounds(seed):
    rng = random.Random(200 + seed)
    c = shape(rng)
    lens = [max(1, n) for n in c["lens"]]
    pool, rows, bounds = K.make(lens, c["hkv"], c["d"], c["dt"], c["bs"], c["fp8"], seed=seed, small=rng.random() < 0.3)
    for _ in range(2):                                     # again: nothing of the first call is counted twice
        want = K.run(pool, rows, bounds, [rng.choice([0, 1, n, rng.randint(0, n)]) for n in lens], lens, rng.choice([0, 9]))
    assert pool.check() == pa.PA_OK and np.isfinite(want[1]).all()
