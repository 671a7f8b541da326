"""The serving operators together: prompts of different lengths are rotated and appended, attended to,
decoded one token further, and a verify of drafts ends in rejection sampling over token distributions."""
import math

import pytest
import torch

from paged_kv_cache_223_gb300 import pagedattn as pa
from serving_reference import adjusted, packed_attention, probs, rotate
from test_gpu_logits import close_adjusted, close_probs
from test_gpu_packed import close

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def step(pool, alloc, rows, lens, new, qkv, hq, hkv, d, rope, scale):
    """Append `new` tokens to each sequence and attend: the block manager's slots, then the two operators."""
    slots, pos = [], []
    for b, n in enumerate(new):
        s, length, copy = alloc.append(rows[b], lens[b], n)
        assert copy is None
        pos += range(lens[b], length)
        slots += s.tolist()
        lens[b] = length
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = pool.rope_append(q, k, v, i32(pos), torch.tensor(slots, device=DEV), rope)
    tables = torch.stack([torch.from_numpy(r.copy()) for r in rows]).to(DEV)
    out = pool.prefill_packed(q, i32(cu), tables, i32(lens), scale)
    return q, out, cu, tables


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_prompts_decode_verify(dt):
    import numpy as np
    hq, hkv, d, bs, V, K = 8, 2, 128, 16, 4000, 3
    g = torch.Generator(device=DEV).manual_seed(5)
    pool = pa.Pool(64, bs, hkv, d, dt, max_seqs=4, max_q_heads=hq, max_context_len=512)
    pool.k_cache.fill_(math.nan), pool.v_cache.fill_(math.nan)
    alloc = pa.BlockAllocator(64, bs)
    inv = [10000.0 ** (-2.0 * i / d) for i in range(d // 2)]
    rope, scale = pa.Rope(inv), 1 / math.sqrt(d)
    rows = [np.zeros(16, np.int32) for _ in range(3)]
    lens = [0, 0, 0]
    past_k = [torch.zeros(0, hkv, d, dtype=torch.float64, device=DEV)] * 3
    for new in ([37, 1, 150], [1, 1, 1], [K + 1] * 3):       # prompts, a decode step, a verify of K drafts
        qkv = torch.randn(sum(new), (hq + 2 * hkv) * d, generator=g, device=DEV).to(dt)
        before = list(lens)
        q, out, cu, tables = step(pool, alloc, rows, lens, new, qkv, hq, hkv, d, rope, scale)
        assert pool.check() == pa.PA_OK
        pos = torch.cat([torch.arange(a, a + n, device=DEV) for a, n in zip(before, new)])
        kref, _ = rotate(qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (-1, d)), pos, inv, False)
        for b in range(3):
            past_k[b] = torch.cat([past_k[b], kref[cu[b]:cu[b + 1]]])
            ids = tables[b, :(lens[b] + bs - 1) // bs].long()
            got = pool.k_cache[ids].permute(0, 2, 1, 3).reshape(-1, hkv, d)[:lens[b]].double()
            assert float((got - past_k[b]).abs().max()) <= float(past_k[b].abs().max()) * torch.finfo(dt).eps
        ref, mag = packed_attention(q, pool.k_cache, pool.v_cache, cu, tables, lens, scale)
        close(out, ref, mag)
        if len(set(new)) == 1 and new[0] <= 4:                # the same tokens through the decode
            i32 = torch.tensor(lens, dtype=torch.int32, device=DEV)
            dec = pool.decode(q.view(3, new[0], hq, d), tables, i32, scale).view(-1, hq, d)
            assert float((dec.double() - out.double()).abs().max()) <= 8 * torch.finfo(dt).eps
    # logits of the verify's rows: a fixed projection of the attention's output
    W = torch.randn(hq * d, V, generator=g, device=DEV).to(dt)
    logits = (out.reshape(3, K + 1, hq * d) @ W)
    draft = torch.randint(0, V, (3, K), generator=g, device=DEV, dtype=torch.int32)
    draft[1, 1] = draft[1, 0]
    hist = torch.randint(0, V, (3, 200), generator=g, device=DEV, dtype=torch.int32)
    kw = dict(history=hist, history_lens=torch.tensor(lens, dtype=torch.int32, device=DEV) - K,
              prompt_lens=torch.tensor([37, 1, 150], dtype=torch.int32, device=DEV), draft=draft,
              repetition=torch.full((3,), 1.2, device=DEV), presence=torch.full((3,), 0.4, device=DEV),
              frequency=torch.full((3,), 0.1, device=DEV))
    kw["mask"] = torch.full((3, K + 1, V // 32), -1, dtype=torch.int32, device=DEV)
    kw["mask"][2, :, :60] = 0
    t = torch.tensor([0.7, 1.0, 0.0], device=DEV)
    p = pa.token_probs(logits, t, **kw)
    ref, mag = adjusted(logits, **kw)
    close_adjusted(pa.adjust_logits(logits, **kw), ref, mag)
    close_probs(p, probs(ref, t), mag, t)
    qd = pa.token_probs((logits[:, :K].float() * 0.5).contiguous(), t.clamp(min=0.7))
    u, v = torch.rand(3, K, generator=g, device=DEV), torch.rand(3, generator=g, device=DEV)
    tok, n = pa.spec_verify(p, qd, draft, u, v)
    import oracle
    want, wn = oracle.spec_verify(*(x.cpu().numpy() for x in (p, qd, draft, u, v)))
    assert n.tolist() == wn.tolist() and tok.tolist() == want.tolist()
    last = tok[2, int(n[2]) - 1]
    assert float(p[2, int(n[2]) - 1, int(last)]) > 0 and int(last) >= 60 * 32
