"""decode_selected: many small weights beside a large one count, in sum and output alike.

Every value is 1; one token of 131072 has a score of 0 (or all of them), all others the same one, of weight w = 2^x: out = (1 + N w) / (1 + N w) =
1. What the product with V loses of the weights is missing from the output: in a warp of 32768 tokens that holds the large one
and loses all of w = 2^-25, 2^-10. Tolerance: the output's rounding, 2^-11, and 4096 weights of 2^-25 lost in a warp or as much
of equal ones by an accumulator's last bit, 2^-13 each: 2^-12."""
import pytest
import torch

from paged_kv_cache_223_gb300 import pagedattn as pa

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("w", [-24.6, -25.05, -26.0, -28.0, 0.0])
def test_many_small_weights_beside_a_large_one(fp8, w):
    B, budget, bs, d = 608, 4096, 32, 128                  # sequences enough to fill the GPU by single CTAs
    pool = pa.Pool(budget, bs, 1, d, torch.float16, max_seqs=1, max_q_heads=1, max_context_len=512,
                   kv_format=pa.PA_KV_FP8_E4M3 if fp8 else pa.PA_KV_16BIT)
    n, scale = budget * bs, 0.001
    x = torch.full((n,), w * 0.6931471805599453 / scale / 16.0)   # times q[0] = 16 and the scale: w in powers of two
    x[0] = 0.0
    if fp8:
        for cache in (pool.k_cache, pool.v_cache):
            cache.zero_()
        pool.k_cache[:n * d].view(n, d)[:, 0] = 0x38          # 1
        pool.k_cache[n * d:].view(torch.float32).copy_(x)
        pool.v_cache[:n * d] = 0x7E                           # 448
        pool.v_cache[n * d:].view(torch.float32).fill_(1 / 448)
    else:
        pool.k_cache.zero_()
        pool.k_cache.view(n, d)[:, 0] = x
        pool.v_cache.fill_(1.0)
    q = torch.zeros(B, 1, 1, d, dtype=torch.float16, device=DEV)
    q[..., 0] = 16.0
    order = torch.arange(budget, dtype=torch.int32, device=DEV)
    tables, sel = order.repeat(B, 1), order.repeat(B, 1, 1)
    out = pool.decode_selected(q, sel, tables, torch.full((B,), n, dtype=torch.int32, device=DEV), scale)
    assert pool.check() == pa.PA_OK
    err = float((out.double() - 1).abs().max())
    assert err <= 2.0 ** -11 + 2.0 ** -12, err
