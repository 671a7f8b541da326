"""The sparse decode step's calls from two threads at once: a kernel's shared memory differs from call to call, and what one
thread asks for must not be lowered by the other's call before it launches."""
import threading

import pytest
import torch

from paged_kv_cache_223_gb300 import pagedattn as pa

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
HQ, HKV, D, BS, NB = 8, 2, 128, 16, 64


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def tables_of(pool, B):
    """One sequence among B gets 20 tokens, over and over."""
    lens, tables = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(B, 4, dtype=torch.int32, device=DEV)
    free, num_free = torch.arange(NB, dtype=torch.int32, device=DEV), i32([NB])
    new, keep = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    new[B - 1] = 20

    def call(stream):
        return pool.step_tables(new, lens, tables, free, num_free, 20, keep_lens=keep, stream=stream)[2]
    return call


def bounds_of(pool, B):
    bounds, lens = pool.new_bounds(), torch.zeros(B, dtype=torch.int32, device=DEV)
    tables, cu = torch.zeros(B, 4, dtype=torch.int32, device=DEV), torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    lens[B - 1] = cu[B] = 20
    tables[B - 1, 1] = 5
    return lambda stream: pool.key_bounds(bounds, cu, tables, lens, 20, stream=stream)


def selection_of(pool, stride):
    bounds, q = pool.new_bounds(), torch.randn(1, 1, HQ, D, dtype=torch.bfloat16, device=DEV)
    tables = torch.zeros(1, stride, dtype=torch.int32, device=DEV)
    tables[0, :40] = torch.arange(40, device=DEV)
    lens = i32([640])
    pool.key_bounds(bounds, i32([0, 640]), tables, lens, 640)
    return lambda stream: pool.select_blocks(q, bounds, tables, lens, 8, stream=stream)


def attention_of(pool, budget):
    q = torch.randn(200, 1, HQ, D, dtype=torch.bfloat16, device=DEV)   # 400 units: few CTAs to a cluster, long lists
    tables = torch.zeros(200, 8, dtype=torch.int32, device=DEV)
    sel = torch.full((200, HKV, budget), -1, dtype=torch.int32, device=DEV)
    sel[:, :, 0] = 0
    lens = torch.full((200,), 16, dtype=torch.int32, device=DEV)
    return lambda stream: pool.decode_selected(q, sel, tables, lens, 0.1, stream=stream)


@pytest.mark.parametrize("make,small,large", [(tables_of, 1, 8000), (bounds_of, 1, 8000), (selection_of, 64, 262144),
                                              (attention_of, 1, 4096)], ids=["tables", "bounds", "selection", "attention"])
def test_two_threads_with_calls_of_different_sizes(make, small, large, monkeypatch):
    pool = pa.Pool(NB, BS, HKV, D, torch.bfloat16, max_seqs=8, max_q_heads=HQ, max_context_len=1024)
    torch.manual_seed(7)
    pool.k_cache.normal_()
    pool.v_cache.normal_()
    calls = [make(pool, small), make(pool, large)]
    want = [call(torch.cuda.current_stream()).clone() for call in calls]
    torch.cuda.synchronize()

    # the C calls with their arguments as the binding makes them: repeated without its checks between them, so that they meet
    streams, outs, ready, one = [torch.cuda.Stream(), torch.cuda.Stream()], [], [], pa._sparse_call
    with monkeypatch.context() as m:
        m.setattr(pa, "_sparse_call", lambda name, *args: (ready.append((pa._sparse_fns[name], args)), one(name, *args)))
        for call, stream in zip(calls, streams):
            outs.append(call(stream))
    torch.cuda.synchronize()
    failed, start = [0, 0], threading.Barrier(2)

    def work(k):
        fn, args = ready[k]
        start.wait()
        for _ in range(15):
            failed[k] += sum(fn(*args) != 0 for _ in range(1000))
            streams[k].synchronize()
    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert failed == [0, 0]
    for out, ref in zip(outs, want):
        assert torch.equal(out.view(torch.uint8), ref.view(torch.uint8))
    assert pool.check() == pa.PA_OK
