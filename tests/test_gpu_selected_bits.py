"""decode_selected on FP8 pools keeps the bits of its weights: where outputs are fp16 they are held as two parts of fp16, so that an
output is off by its own rounding and what 32-bit sums lose, not by 2^-11 of the weights as well.

Tolerance of an output:
- its own rounding, eps / 2 of the value;
- relative to sum p |v|: weights of two parts 2^-21 (of one, FP8 pools with bf16 outputs, 2^-11:
  half a step of fp16), exponentials and sums of 32 bits
  2^-20, a score's sum of products (of size `big`, in units of e) 2^-20 big and as much for the reference's terms, and one unit
  in the last place for each of a warp's additions, N / 16 in all at most: N 2^-26;
- a weight is lost whole, or off by the last bit that its type holds: the sum of min(p, 2^-28) |v| (of one part 2^-25).
"""
import math

import pytest
import torch

from paged_kv_cache_223_gb300 import pagedattn as pa
from test_gpu_decode_selected import i32, make, pick, reader

pytestmark = pytest.mark.gpu


def definition(pool, q, selected, tables, lens, scale):
    """The output in 64 bits and its tolerance, [B, n, Hq, d] each."""
    keys, values = reader(pool, pool.k_cache, tables), reader(pool, pool.v_cache, tables)
    (B, n, hq, d), hkv, bs, dt = q.shape, selected.shape[1], pool.geometry[2], torch.finfo(q.dtype)
    two = not (pool.kv_format == pa.PA_KV_FP8_E4M3 and q.dtype == torch.bfloat16)
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    N = selected.shape[2] * bs
    for b in range(B):
        for h in range(hkv):
            js = [j for j in selected[b, h].tolist() if j >= 0]
            if not js:
                continue
            k, v = (torch.cat([x(b, h, j) for j in js]) for x in (keys, values))
            pos = torch.cat([torch.arange(j * bs, (j + 1) * bs, device=q.device) for j in js])
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            for r in range(n):
                seen = (pos <= lens[b] - n + r).nonzero()[:, 0]
                if seen.numel():
                    x, ks, vs = q[b, r, heads].double(), k[seen], v[seen]
                    size = vs.abs().nan_to_num(0.0, 0.0, 0.0)
                    p = torch.softmax(x @ ks.T * scale, -1)
                    out[b, r, heads] = p @ vs
                    rel = (2.0 ** -21 if two else 2.0 ** -11) + 2.0 ** -20 + N * 2.0 ** -26
                    big = (x.abs() @ ks.abs().T).amax(-1, keepdim=True) * abs(scale)
                    tol[b, r, heads] = (p @ size) * (rel + big * 2.0 ** -19) + p.clamp(max=2.0 ** (-28 if two else -25)) @ size
    return out, tol + out.abs().nan_to_num(0.0, 0.0, 0.0) * dt.eps / 2 + dt.smallest_normal * dt.eps / 2


def run(pool, tables, q, lens, selected, scale=None):
    """The output, where numbers are expected within their tolerance; elsewhere the same infinity or NaN (what is beyond the type's
    largest number rounds to an infinity)."""
    scale = 1 / math.sqrt(pool.geometry[3]) if scale is None else scale
    got = pool.decode_selected(q, selected, tables, i32(lens), scale)
    out, tol = definition(pool, q, selected, tables, lens, scale)
    most = torch.finfo(q.dtype).max
    number, odd = out.abs() + tol < most, ~(out.abs() - tol.nan_to_num(0.0) < most * (1 + torch.finfo(q.dtype).eps))
    sign = lambda x: x.nan_to_num(0.0, math.inf, -math.inf).sign()  # noqa: E731
    assert torch.equal(got[odd].isnan(), out[odd].isnan()) and torch.equal(sign(got[odd].double()), sign(out[odd]))
    assert not bool(got[odd].isfinite().any())
    worst = float(((got.double() - out).abs() / tol)[number].nan_to_num(math.inf).max())
    assert worst <= 1, f"{worst:.3g} of the tolerance"
    assert pool.check() == pa.PA_OK
    return got


@pytest.mark.parametrize("lens,hq,hkv,bs,q_len,budget", [
    ([1], 4, 4, 16, 1, 2),
    ([500, 33, 64], 32, 8, 32, 1, 6),
    ([700, 90, 6], 8, 2, 16, 4, 20),                       # 16 rows
    ([900, 40], 12, 2, 32, 4, 12),                         # 24
    ([1500, 31], 32, 1, 16, 1, 60),                        # 32
])
def test_weights_in_two_parts(lens, hq, hkv, bs, q_len, budget):
    """fp16 outputs, whose rounding is 2^-11: weights of one part would add half of it."""
    pool, tables, q = make(lens, hq, hkv, 128, torch.float16, bs, q_len, fp8=True, seed=budget)
    run(pool, tables, q, lens, pick(lens, hkv, bs, budget, 2))


@pytest.mark.parametrize("dt,fp8", [(torch.float16, True), (torch.bfloat16, True), (torch.float16, False), (torch.bfloat16, False)])
def test_weighted_values_that_cancel(dt, fp8):
    """Values of both signs whose weighted sum is small beside them: the weights' error is not hidden by the output's
    rounding."""
    lens = [320]
    pool, tables, q = make(lens, 8, 2, 128, dt, 16, 2, fp8=fp8, seed=3)
    if fp8:
        n = pool.geometry[0] * 2 * 16 * 128
        codes, scales = pool.v_cache[:n].view(-1, 128), pool.v_cache[n:].view(torch.float32)
        codes[1::2] = codes[::2] ^ 0x80                    # each second token is the one before it, negated
        scales[1::2] = scales[::2]
    else:
        pool.v_cache[:, :, 1::2] = -pool.v_cache[:, :, ::2]
    q *= 0.02                                              # nearly equal weights
    run(pool, tables, q, lens, pick(lens, 2, 16, 20, 4))
