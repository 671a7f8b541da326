"""A whole sparse decode step in one graph (tables, rotation and append, bounds, selection, attention), replayed token after token
across block ends: bit for bit what the same calls give one by one on a pool of their own."""
import math

import pytest
import torch

from paged_kv_cache_223_gb300 import pagedattn as pa

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
HQ, HKV, B, NB, STRIDE = 8, 2, 3, 120, 40


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Loop:
    def __init__(self, dt, d, bs, fp8):
        self.pool = pa.Pool(NB, bs, HKV, d, dt, max_seqs=B, max_q_heads=HQ, max_context_len=STRIDE * bs,
                            kv_format=pa.PA_KV_FP8_E4M3 if fp8 else pa.PA_KV_16BIT)
        for c in (self.pool.k_cache, self.pool.v_cache):
            c.view(torch.uint8).zero_()
        self.d, self.rope, self.bounds = d, pa.Rope.from_base(d), self.pool.new_bounds()
        self.state = dict(context_lens=i32([0] * B), block_tables=torch.full((B, STRIDE), -1, dtype=torch.int32, device=DEV),
                          free_blocks=torch.arange(NB, dtype=torch.int32, device=DEV), num_free=i32([NB]))

    def step(self, new, keep, qkv):
        """One step of the tokens of qkv; of a token for each sequence the attention's output too."""
        n, s = qkv.shape[0], self.state
        cu, pos, slots = self.pool.step_tables(new, num_tokens=n, keep_lens=keep, **s)
        q, k, v = (x.unflatten(1, (-1, self.d)) for x in qkv.split([HQ * self.d, HKV * self.d, HKV * self.d], 1))
        q = self.pool.rope_append(q, k, v, pos, slots, self.rope)
        self.pool.key_bounds(self.bounds, cu, s["block_tables"], s["context_lens"], n)
        if n != B:
            return cu, pos, slots
        q = q.view(B, 1, HQ, self.d)
        sel = self.pool.select_blocks(q, self.bounds, s["block_tables"], s["context_lens"], 7)
        return cu, pos, slots, sel, self.pool.decode_selected(q, sel, s["block_tables"], s["context_lens"], 1 / math.sqrt(self.d))

    def all(self):
        return [*self.state.values(), self.bounds, self.pool.k_cache, self.pool.v_cache]


@pytest.mark.parametrize("dt,d,bs,fp8", [(torch.bfloat16, 128, 16, False), (torch.float16, 64, 32, False), (torch.float16, 128, 16, True)])
def test_a_captured_step(dt, d, bs, fp8):
    g = torch.Generator(device=DEV).manual_seed(bs + d)
    captured, single = Loop(dt, d, bs, fp8), Loop(dt, d, bs, fp8)
    rand = lambda n: torch.randn(n, (HQ + 2 * HKV) * d, generator=g, device=DEV).to(dt)  # noqa: E731
    new, keep = i32([300, 61, 130]), i32([2 ** 30] * B)
    prompts = rand(491)
    for loop in (captured, single):
        loop.step(new, keep, prompts)
    one, qkv = i32([1] * B), rand(B)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = captured.step(one, keep, qkv)
    for i in range(40):
        qkv.copy_(rand(B))
        keep.fill_(2 ** 30)
        if i == 9:
            keep[0] = 290                                  # tokens cut between two replays
        graph.replay()
        for got, want in zip([*outs, *captured.all()], [*single.step(one, keep, qkv), *single.all()]):
            assert torch.equal(got.view(torch.uint8), want.view(torch.uint8)), i
    assert captured.state["context_lens"].tolist() == [290 + 31, 101, 170]
    assert captured.pool.check() == pa.PA_OK and single.pool.check() == pa.PA_OK
