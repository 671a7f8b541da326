"""A sparse decode loop of all its calls: tables on the device, rotation and append, bounds, selection, attention."""
import math

import numpy as np
import pytest
import torch

from paged_kv_cache_223_gb300 import pagedattn as pa
from sparse_reference import step_tables
from test_gpu_decode_selected import close, reference
from test_gpu_key_bounds import expected as expected_bounds
from test_gpu_key_bounds import parts
from test_gpu_select_blocks import expected as expected_selection

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dt,d,bs,fp8", [(torch.bfloat16, 128, 16, False), (torch.float16, 64, 32, False),
                                         (torch.bfloat16, 128, 32, True)])
def test_prompts_then_steps(dt, d, bs, fp8):
    B, hq, hkv, nb, stride, budget = 4, 8, 2, 200, 64, 9
    g = torch.Generator(device=DEV).manual_seed(d + bs)
    pool = pa.Pool(nb, bs, hkv, d, dt, max_seqs=B, max_q_heads=hq, max_context_len=stride * bs,
                   kv_format=pa.PA_KV_FP8_E4M3 if fp8 else pa.PA_KV_16BIT)
    pool.k_cache.view(torch.uint8).fill_(0x7F), pool.v_cache.view(torch.uint8).fill_(0x7F)
    rope, scale, bounds = pa.Rope.from_base(d), 1 / math.sqrt(d), pool.new_bounds()
    state = dict(context_lens=i32([0] * B), block_tables=torch.full((B, stride), -1, dtype=torch.int32, device=DEV),
                 free_blocks=torch.randperm(nb, generator=g, device=DEV).to(torch.int32), num_free=i32([nb]))
    lens, rows, free, num_free = [0] * B, state["block_tables"].tolist(), state["free_blocks"].tolist(), nb
    # prompts; a token each; a verify of two drafts; drafts rejected and an ended request's place taken by a prompt; a token
    steps = [([500, 37, 0, 260], None), ([1, 1, 0, 1], None), ([3, 3, 0, 3], None), ([1, 1, 90, 77], [502, 10 ** 9, 0, 0]),
             ([1, 1, 1, 1], None), ([1, 1, 1, 1], None)]
    for new, keep in steps:
        total = sum(new) + 2
        cu, pos, slots = pool.step_tables(i32(new), num_tokens=total, keep_lens=None if keep is None else i32(keep), **state)
        rows, lens, free, num_free, hcu, hpos, hslots = step_tables(new, lens, rows, free, num_free, total, bs, keep)
        assert (cu.tolist(), pos.tolist(), slots.tolist()) == (hcu, hpos, hslots)
        assert state["context_lens"].tolist() == lens and state["block_tables"].tolist() == rows
        qkv = torch.randn(total, (hq + 2 * hkv) * d, generator=g, device=DEV).to(dt)
        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
        q = pool.rope_append(q, k, v, pos, slots, rope)
        want = expected_bounds(pool, bounds, hcu, rows, lens)
        pool.key_bounds(bounds, cu, state["block_tables"], state["context_lens"], total)
        codes, sizes = parts(pool, bounds)
        assert np.array_equal(codes.cpu().numpy(), want[0]) and np.array_equal(sizes.cpu().numpy(), want[1])
        assert pool.check() == pa.PA_OK
        n = max(new)
        if n > 3 or min(m for m in new if m) != n:
            continue                                       # prompts: not this call's
        live = [b for b in range(B) if new[b]]
        at = torch.tensor([hcu[b] for b in live], device=DEV)[:, None] + torch.arange(n, device=DEV)
        q = q[at].contiguous()
        tables, dl, hl = state["block_tables"][live].contiguous(), i32([lens[b] for b in live]), [lens[b] for b in live]
        sel = pool.select_blocks(q, bounds, tables, dl, budget)
        assert np.array_equal(sel.cpu().numpy(), expected_selection(q, codes.long(), sizes, tables, hl, bs, budget, 1, 2))
        out = pool.decode_selected(q, sel, tables, dl, scale)
        close(out, reference(pool, q, sel, tables, hl, scale), sel, bs, fp8, 6.0)
        every = pool.select_blocks(q, bounds, tables, dl, stride)        # room for all: the whole context
        dense, whole = pool.decode(q, tables, dl, scale), pool.decode_selected(q, every, tables, dl, scale)
        assert float((dense.double() - whole.double()).abs().max()) <= 4 * torch.finfo(dt).eps * float(dense.abs().max())
        assert pool.check() == pa.PA_OK
