"""decode_selected on FP8 pools whose V scales lie far apart: a token that hardly counts takes no bits from those that do,
whatever its scale is. Tolerances are relative to what each token adds to its row, never to the largest scale."""
import pytest
import torch

from test_gpu_decode_selected import make, pick
from test_gpu_selected_bits import run

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def parts(pool, cache):
    nb, hkv, bs, d = pool.geometry
    return cache[:nb * hkv * bs * d].view(nb, hkv, bs, d), cache[nb * hkv * bs * d:].view(torch.float32).view(nb, hkv, bs)


def far(pool, tables, q, b, token, power):
    """A token of sequence b with a weight below 2^-60 and a V scale 2^power times as large."""
    bs = pool.geometry[2]
    block = int(tables[b, token // bs])
    codes, scales = parts(pool, pool.k_cache)
    q[b, ..., 0] = 8.0
    codes[block, :, token % bs] = 0
    codes[block, :, token % bs, 0] = 0xFE                  # -448
    scales[block, :, token % bs] = 1.0                     # a score of -3584 times the softmax scale
    parts(pool, pool.v_cache)[1][block, :, token % bs] *= 2.0 ** power


@pytest.mark.parametrize("dt,hq,q_len", [(torch.float16, 8, 1), (torch.bfloat16, 16, 2), (torch.float16, 24, 2),
                                         (torch.bfloat16, 32, 2)])
@pytest.mark.parametrize("power", [14, 18, 20, 25, 40, 90])
@pytest.mark.parametrize("token", [0, 250, 503])
def test_a_large_scale_without_weight(dt, hq, q_len, power, token):
    lens = [512, 100]
    pool, tables, q = make(lens, hq, 2, 128, dt, 16, q_len, fp8=True, seed=hq)
    sel = pick(lens, 2, 16, 32, 2)
    far(pool, tables, q, 0, token, power)
    run(pool, tables, q, lens, sel)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("budget", [1, 6, 60])
def test_scales_of_any_order(dt, budget):
    """Scales 2^36 apart, in no order and by stretches of tokens; so are they among the tokens that not every row sees."""
    lens = [900, 70, 18]
    pool, tables, q = make(lens, 8, 2, 128, dt, 16, 4, fp8=True, seed=budget)
    sel = pick(lens, 2, 16, budget, 3)
    scales = parts(pool, pool.v_cache)[1]
    base = scales.clone()
    g = torch.Generator(device=DEV).manual_seed(budget)
    scales.copy_(base * torch.exp2(torch.randint(-18, 19, base.shape, generator=g, device=DEV).float()))
    run(pool, tables, q, lens, sel)
    scales.copy_(base * torch.exp2(torch.randint(-18, 19, base.shape[:2] + (1,), generator=g, device=DEV).float()))
    run(pool, tables, q, lens, sel)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("power", [-30, -14, -7, 7, 14])
def test_rows_of_zeros_and_of_another_size(dt, power):
    """What a cache holds in earnest: rows of zeros, stored with a scale of 1 or 0, and a few rows of another size."""
    lens = [640, 31]
    pool, tables, q = make(lens, 8, 2, 128, dt, 16, 1, fp8=True, seed=5, vscale=2.0 ** (-4 if dt == torch.float16 else -12))
    codes, scales = parts(pool, pool.v_cache)
    codes[:, :, 3], scales[:, :, 3] = 0, 1.0
    codes[:, :, 4], scales[:, :, 4] = 0, 0.0
    scales[::7, :, 11] *= 2.0 ** power
    run(pool, tables, q, lens, pick(lens, 2, 16, 40, 4))


@pytest.mark.parametrize("dt", [torch.bfloat16])
@pytest.mark.parametrize("power", [-100, -80, 90, 100])
def test_scales_at_the_ends_of_their_range(dt, power):
    lens = [300, 17]
    pool, tables, q = make(lens, 8, 2, 128, dt, 16, 2, fp8=True, seed=6)
    parts(pool, pool.v_cache)[1].mul_(2.0 ** power)
    run(pool, tables, q, lens, pick(lens, 2, 16, 19, 5))
