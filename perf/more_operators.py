"""Measured cases of the operators of a sparse decode step on the paged cache: step_tables (block tables,
positions and slots from request lengths), key_bounds (the bounds of each block's keys), select_blocks
(the blocks that a cheap score picks for each query) and decode_selected (attention over them).

With `own` false, run() computes each operator in its plain form (elementary torch operations in 32
bits, whole numbers as such); with `own` true it calls the library. prepare() makes the inputs from the
seed and what a serving program keeps: the pool's handle, the free list, the bounds of the cache.
"""
import math
import random

import torch

own = False

_DTYPE = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # step_tables: one request takes one more token
        dict(name="tables-1", op="tables", b=1, new_lo=1, new_hi=1, cut=0, old_lo=700, old_hi=700, ended=0, mix=1, bs=16,
             pad=0, spare=32),
        # step_tables: a decode step of a large batch behind a verify: up to five rejected tokens are taken back, some
        # requests have ended and make room for new prompts
        dict(name="tables-verify-257", op="tables", b=257, new_lo=1, new_hi=6, cut=5, old_lo=100, old_hi=8192, ended=12,
             mix=2, bs=16, pad=64, spare=1000),
        # step_tables: many prompts at once, of very different lengths
        dict(name="tables-prompts-2000", op="tables", b=2000, new_lo=1, new_hi=1024, cut=0, old_lo=1, old_hi=4096,
             ended=1000, mix=3, bs=32, pad=1, spare=40000),
        # key_bounds: a decode step, one new token in the last block of each sequence
        dict(name="bounds-decode-64", op="bounds", b=64, new_lo=1, new_hi=1, old_lo=100, old_hi=300, mix=4, hkv=8, d=128,
             dtype="bf16", fp8=False, bs=16),
        # key_bounds: the blocks of a step of prompts
        dict(name="bounds-prompts-5", op="bounds", b=5, new_lo=1500, new_hi=6000, old_lo=0, old_hi=100, mix=5, hkv=8,
             d=128, dtype="fp16", fp8=False, bs=16),
        # key_bounds: an 8-bit pool, odd lengths
        dict(name="bounds-fp8-33", op="bounds", b=33, new_lo=3, new_hi=700, old_lo=0, old_hi=500, mix=6, hkv=8, d=128,
             dtype="bf16", fp8=True, bs=32),
        # select_blocks: one sequence with a long context
        dict(name="select-1x131072", op="select", b=1, ctx_lo=131072, ctx_hi=131072, q_len=1, hq=32, hkv=8, d=128,
             dtype="bf16", bs=16, budget=128, first=1, last=4, mix=7),
        # select_blocks: a decode step of a batch, the largest call
        dict(name="select-64x16384", op="select", b=64, ctx_lo=15000, ctx_hi=16384, q_len=1, hq=64, hkv=8, d=128,
             dtype="bf16", bs=16, budget=128, first=1, last=4, mix=8),
        # select_blocks: a verify of four drafts, small heads, contexts from a few tokens to long ones
        dict(name="select-verify-13", op="select", b=13, ctx_lo=40, ctx_hi=60000, q_len=5, hq=20, hkv=4, d=64,
             dtype="fp16", bs=32, budget=65, first=2, last=3, mix=9),
        # decode_selected: one sequence, where latency counts
        dict(name="attend-1", op="attend", b=1, ctx_lo=32768, ctx_hi=32768, q_len=1, hq=32, hkv=8, d=128, dtype="bf16",
             fp8=False, bs=16, budget=64, mix=10),
        # decode_selected: a decode step of a batch, the largest call
        dict(name="attend-64", op="attend", b=64, ctx_lo=4000, ctx_hi=8192, q_len=1, hq=64, hkv=8, d=128, dtype="bf16",
             fp8=False, bs=16, budget=128, mix=11),
        # decode_selected: a verify of three drafts on an 8-bit pool, some contexts shorter than the budget
        dict(name="attend-fp8-verify-19", op="attend", b=19, ctx_lo=90, ctx_hi=20000, q_len=4, hq=32, hkv=8, d=128,
             dtype="fp16", fp8=True, bs=32, budget=50, mix=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "bounds", "select", "attend"])
    mix, bs = rng.randrange(1, 1000000), rng.choice([16, 32])
    if op == "tables":
        while True:
            new_hi = _log(rng, 1, 4096)
            c = dict(op="tables", b=_log(rng, 1, 2000), new_lo=rng.choice([0, 1, new_hi]), new_hi=new_hi,
                     cut=rng.choice([0, 0, 5, 100]), old_lo=rng.choice([0, 1]), old_hi=_log(rng, 1, 8192), ended=0, mix=mix,
                     bs=bs, pad=rng.choice([0, 1, 100]), spare=_log(rng, 1, 1000))
            c["ended"] = rng.randint(0, c["b"] // 2)
            if c["b"] * new_hi <= 2 ** 19 and c["b"] * c["old_hi"] <= 2 ** 23:
                return c
    hq, hkv = rng.choice([(32, 8), (64, 8), (16, 16), (8, 1), (20, 4), (12, 4)])
    dtype, d = rng.choice(["bf16", "fp16"]), rng.choice([64, 128, 128])
    if op == "bounds":
        while True:
            new_hi = _log(rng, 1, 8192)
            c = dict(op="bounds", b=_log(rng, 1, 256), new_lo=rng.choice([1, new_hi]), new_hi=new_hi, old_lo=0,
                     old_hi=rng.choice([0, _log(rng, 1, 500)]), mix=mix, hkv=hkv, d=d, dtype=dtype,
                     fp8=d == 128 and rng.random() < 0.3, bs=bs)
            if c["b"] * (c["new_hi"] + c["old_hi"] + bs) * hkv * d <= 16384 * 1024:
                return c
    while True:
        q_len = rng.choice([1, 1, 2, 4, 5, 8])
        ctx_hi = _log(rng, 20, 131072)
        c = dict(op=op, b=_log(rng, 1, 64), ctx_lo=rng.choice([ctx_hi, max(8, ctx_hi // 50), max(8, ctx_hi // 2)]),
                 ctx_hi=ctx_hi, q_len=q_len, hq=hq, hkv=hkv, d=d, dtype=dtype, bs=bs, budget=_log(rng, 4, 256), mix=mix)
        tokens = c["b"] * min(ctx_hi, c["budget"] * bs) * hkv * d
        if q_len * hq // hkv > 32 or c["b"] * ctx_hi * hkv * d > 64 * 16384 * 1024 // 2:
            continue
        if op == "attend":
            c["fp8"] = d == 128 and rng.random() < 0.3
            if tokens <= 64 * 2048 * 1024:
                return c
        else:
            c["first"], c["last"] = rng.choice([0, 1, 2]), 2
            # a selection that leaves something out
            if c["budget"] >= 8 and _blocks(max(_lens(c)), bs) >= 2 * c["budget"]:
                return c


def _spread(rng, n, lo, hi):
    """n lengths between lo and hi, spread over the logarithm; where lo is 0, about one in hi + 1 of them is."""
    return [0 if lo == 0 and rng.random() * (hi + 1) < 1 else _log(rng, max(lo, 1), hi) for _ in range(n)]


def _lens(case):
    """The lengths of a case's sequences, fixed by the case. tables: old, kept and new; bounds: old and new; else: contexts."""
    rng = random.Random(case["mix"])
    b = case["b"]
    if case["op"] in ("select", "attend"):
        return _spread(rng, b, case["ctx_lo"], case["ctx_hi"])
    old, new = _spread(rng, b, case["old_lo"], case["old_hi"]), _spread(rng, b, case["new_lo"], case["new_hi"])
    if case["op"] == "bounds":
        return old, new
    kept = [max(0, n - rng.randint(0, case["cut"])) for n in old]
    for i in rng.sample(range(b), case["ended"]):
        kept[i] = 0
    return old, kept, new


def _blocks(n, bs):
    return (n + bs - 1) // bs


def work(case):
    bs = case["bs"]
    if case["op"] == "tables":
        old, kept, new = _lens(case)
        back = sum(_blocks(o, bs) - _blocks(k, bs) for o, k in zip(old, kept))
        taken = sum(_blocks(k + n, bs) - _blocks(k, bs) for k, n in zip(kept, new))
        tokens = sum(new) + case["pad"]
        return {"bytes": case["b"] * 20 + tokens * 12 + (back + taken) * 8, "flops": tokens * 4}
    d, hkv = case["d"], case["hkv"]
    if case["op"] == "bounds":
        old, new = _lens(case)
        first = [o // bs * bs for o in old]
        rows = sum(o + n - f for o, n, f in zip(old, new, first))
        blocks = sum(_blocks(o + n - f, bs) for o, n, f in zip(old, new, first))
        return {"bytes": hkv * (rows * (d + 4 if case["fp8"] else 2 * d) + blocks * (2 * d + 4)) + blocks * 4,
                "flops": 2 * rows * hkv * d}
    lens, rows = _lens(case), case["q_len"] * case["hq"]
    blocks = [_blocks(n, bs) for n in lens]
    if case["op"] == "select":
        return {"bytes": sum(blocks) * (hkv * (2 * d + 4) + 4) + case["b"] * (rows * d * 2 + hkv * case["budget"] * 4),
                "flops": 4 * d * rows * sum(blocks)}
    tokens = sum(min(n, min(m, case["budget"]) * bs) for n, m in zip(lens, blocks))
    return {"bytes": tokens * hkv * 2 * (d + 4 if case["fp8"] else 2 * d) + case["b"] * rows * d * 4 +
            sum(min(m, case["budget"]) for m in blocks) * (hkv + 1) * 4, "flops": 4 * d * rows * tokens}


# ----------------------------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"tables": _prepare_tables, "bounds": _prepare_bounds, "select": _prepare_select,
            "attend": _prepare_attend}[case["op"]](dict(case), g)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _pool(s, nb, **kw):
    if own:
        from paged_kv_cache_223_gb300 import pagedattn as pa
        kw.setdefault("kv_format", pa.PA_KV_FP8_E4M3 if s.get("fp8") else pa.PA_KV_16BIT)
        s["pool"] = pa.Pool(nb, s["bs"], s.get("hkv", 1), s.get("d", 64), dtype=_DTYPE[s.get("dtype", "fp16")], max_seqs=1,
                            max_q_heads=s.get("hq", 1), max_q_len=s.get("q_len", 1), max_context_len=512, **kw)


def _tables(s, g, blocks, nb):
    """A table row of distinct blocks for each sequence, and the ids that are left."""
    ids = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    stride = max(max(blocks), 1)
    tables = torch.zeros(len(blocks), stride, dtype=torch.int32, device="cuda")
    count = torch.tensor(blocks, device="cuda")
    tables[torch.arange(stride, device="cuda")[None, :] < count[:, None]] = ids[:sum(blocks)]
    return tables, ids[sum(blocks):]


def _prepare_tables(s, g):
    old, kept, new = _lens(s)
    bs = s["bs"]
    have = [_blocks(n, bs) for n in old]
    need = [max(h, _blocks(k + n, bs)) for h, k, n in zip(have, kept, new)]
    nb = sum(need) + s["spare"]
    tables, free = _tables(s, g, have, nb)
    s["block_tables"] = torch.nn.functional.pad(tables, (0, max(1, max(need)) - tables.shape[1]), value=-1)
    s["free"] = torch.full((nb,), -1, dtype=torch.int32, device="cuda")
    s["free"][:free.numel()] = free
    s["num_free"] = _i32([free.numel()])
    s["lens"], s["keep"], s["new"] = _i32(old), _i32(kept), _i32(new)
    s["num_tokens"] = sum(new) + s["pad"]
    _pool(s, nb)
    return s


def _cache(g, s, nb):
    """One cache of keys or values, whose channels differ in size; an 8-bit one as codes followed by scales."""
    hkv, bs, d = s["hkv"], s["bs"], s["d"]
    x = _randn(g, nb, hkv, bs, d).mul_(1.0 + _randn(g, 1, hkv, 1, d).abs_())
    if not s["fp8"]:
        return x.to(_DTYPE[s["dtype"]])
    scale = x.abs().amax(-1) / 448.0
    codes = (x / scale[..., None]).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.cat([codes.view(-1), scale.view(-1).view(torch.uint8)])


def _prepare_bounds(s, g):
    old, new = _lens(s)
    bs, hkv, d = s["bs"], s["hkv"], s["d"]
    blocks = [_blocks(o + n, bs) for o, n in zip(old, new)]
    nb = sum(blocks) + 3
    s["nb"] = nb
    s["k_cache"] = _cache(g, s, nb)
    s["block_tables"], _ = _tables(s, g, blocks, nb)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["cu_q"], s["lens"] = _i32(cu), _i32([o + n for o, n in zip(old, new)])
    s["num_tokens"] = cu[-1]
    s["touched"] = sum(m - o // bs for m, o in zip(blocks, old))
    # what an earlier step left
    codes = torch.randint(-127, 128, (nb * hkv * 2 * d,), generator=g, device="cuda", dtype=torch.int16).to(torch.int8)
    steps = torch.exp2(torch.randint(-8, 0, (nb * hkv,), generator=g, device="cuda").float())
    s["bounds"] = torch.cat([codes.view(torch.uint8), steps.view(torch.uint8)])
    _pool(s, nb, k_cache=s["k_cache"], v_cache=s["k_cache"])
    return s


def _step(top):
    """The smallest power of two s with top <= 127 s (0 for 0): built from its exponent, exact for normal numbers."""
    m, e = torch.frexp(top)
    e = e - 7 + (m > 127.0 / 128.0).to(torch.int32)
    return torch.where(top > 0, ((e + 127) << 23).view(torch.float32), torch.zeros_like(top))


def _codes(x, step):
    """Nearest whole multiples of step (ties to even), a power of two: exact."""
    return torch.round(x / torch.where(step > 0, step, torch.ones_like(step)))


def _prepare_select(s, g):
    lens = _lens(s)
    bs, hkv, d = s["bs"], s["hkv"], s["d"]
    blocks = [_blocks(n, bs) for n in lens]
    nb = sum(blocks) + 3
    s["nb"] = nb
    s["block_tables"], _ = _tables(s, g, blocks, nb)
    s["lens"] = _i32(lens)
    # blocks' keys lie around a middle of their own, channels differ in size
    size = 1.0 + _randn(g, 1, hkv, d).abs_()
    middle, half = _randn(g, nb, hkv, d).mul_(size * 0.6), _randn(g, nb, hkv, d).mul_(0.3).add_(1.7).mul_(size)
    hi, lo = middle + half, middle - half
    step = _step(torch.maximum(hi.abs(), lo.abs()).amax(-1))
    codes = _codes(torch.stack([hi, lo], 2), step[..., None, None]).to(torch.int8)
    s["bounds"] = torch.cat([codes.view(-1).view(torch.uint8), step.view(-1).view(torch.uint8)])
    s["q"] = _randn(g, s["b"], s["q_len"], s["hq"], d).to(_DTYPE[s["dtype"]])
    if own:
        kv = torch.empty(nb, hkv, bs, d, dtype=_DTYPE[s["dtype"]], device="cuda")
        _pool(s, nb, k_cache=kv, v_cache=kv)
    return s


def _prepare_attend(s, g):
    lens = _lens(s)
    bs, hkv, budget = s["bs"], s["hkv"], s["budget"]
    blocks = [_blocks(n, bs) for n in lens]
    nb = sum(blocks) + 3
    s["nb"] = nb
    s["k_cache"], s["v_cache"] = _cache(g, s, nb), _cache(g, s, nb)
    s["block_tables"], _ = _tables(s, g, blocks, nb)
    s["lens"] = _i32(lens)
    s["q"] = (_randn(g, s["b"], s["q_len"], s["hq"], s["d"]) * 0.7).to(_DTYPE[s["dtype"]])
    s["scale"] = 1.0 / math.sqrt(s["d"])
    # the blocks that a selection leaves: the first, the last and others anywhere, ascending, -1 behind them
    order = torch.rand(s["b"], hkv, max(blocks), generator=g, device="cuda")
    at = torch.arange(max(blocks), device="cuda")
    count = torch.tensor(blocks, device="cuda")[:, None, None]
    order = torch.where((at == 0) | (at == count - 1), -1.0, order).masked_fill(at >= count, 2.0)
    value, pick = order.topk(min(budget, max(blocks)), dim=-1, largest=False)
    pick = pick.masked_fill(value >= 2.0, 2 ** 30).sort(-1).values
    pick = torch.where(pick < 2 ** 30, pick, -1).to(torch.int32)
    s["selected"] = torch.nn.functional.pad(pick, (0, budget - pick.shape[-1]), value=-1).contiguous()
    _pool(s, nb, k_cache=s["k_cache"], v_cache=s["v_cache"])
    return s


# ------------------------------------------------------------------------------------ one pass

def run(s):
    return {"tables": _run_tables, "bounds": _run_bounds, "select": _run_select, "attend": _run_attend}[s["op"]](s)


def _run_tables(s):
    if own:
        cu_q, positions, slots = s["pool"].step_tables(s["new"], s["lens"], s["block_tables"], s["free"], s["num_free"],
                                                       s["num_tokens"], keep_lens=s["keep"])
        return s["block_tables"], s["lens"], s["free"], s["num_free"], cu_q, positions, slots
    bs, tables, free = s["bs"], s["block_tables"], s["free"]
    b, stride = tables.shape
    kept = torch.minimum(s["lens"], s["keep"])
    have, old = (kept + bs - 1) // bs, (s["lens"] + bs - 1) // bs
    length = kept + s["new"]
    want = torch.maximum(have, (length + bs - 1) // bs)
    back, taken = (old - have).cumsum(0), (want - have).cumsum(0)
    top = s["num_free"] + back[-1]
    at = torch.arange(stride, dtype=torch.int32, device="cuda")[None, :]
    # blocks that are given back: the first one ends on top
    gone = (at >= have[:, None]) & (at < old[:, None])
    place = top - 1 - ((back - (old - have))[:, None] + at - have[:, None])
    place = torch.where(gone, place, free.numel()).long()
    free.copy_(torch.cat([free, free[:1]]).scatter_(0, place.view(-1), tables.reshape(-1))[:-1])
    # blocks that are taken, from the top
    fresh = (at >= have[:, None]) & (at < want[:, None])
    place = top - 1 - ((taken - (want - have))[:, None] + at - have[:, None])
    tables.copy_(torch.where(fresh, free[torch.where(fresh, place, 0).long()], tables))
    s["num_free"].copy_(top - taken[-1])
    cu_q = torch.cat([torch.zeros_like(kept[:1]), s["new"].cumsum(0, dtype=torch.int32)])
    tok = torch.arange(s["num_tokens"], dtype=torch.int32, device="cuda")
    seq = torch.searchsorted(cu_q[1:], tok, right=True).clamp_(max=b - 1)
    live = tok < cu_q[-1]
    positions = torch.where(live, kept[seq] + tok - cu_q[seq], 0)
    slots = torch.where(live, tables[seq, (positions // bs).long()].long() * bs + positions % bs, -1)
    s["lens"].copy_(length)
    return tables, s["lens"], free, s["num_free"], cu_q, positions, slots


def _values(cache, s):
    """A cache's values in 32 bits, [nb, hkv, bs, d]; of an 8-bit one code * scale."""
    shape = (s["nb"], s["hkv"], s["bs"], s["d"])
    if not s["fp8"]:
        return cache.float()
    n = math.prod(shape)
    return cache[:n].view(torch.float8_e4m3fn).float().view(shape) * cache[n:].view(torch.float32).view(shape[:3])[..., None]


def _bounds_of(s):
    """The bounds buffer's parts: codes [nb, hkv, 2, d] (upper, lower) and steps [nb, hkv]."""
    n = s["nb"] * s["hkv"] * 2 * s["d"]
    return (s["bounds"][:n].view(torch.int8).view(s["nb"], s["hkv"], 2, s["d"]),
            s["bounds"][n:].view(torch.float32).view(s["nb"], s["hkv"]))


def _run_bounds(s):
    codes, steps = _bounds_of(s)
    if own:
        s["pool"].key_bounds(s["bounds"], s["cu_q"], s["block_tables"], s["lens"], s["num_tokens"])
    else:
        bs = s["bs"]
        first = (s["lens"] - (s["cu_q"][1:] - s["cu_q"][:-1])) // bs
        count = (s["lens"] + bs - 1) // bs - first
        seq = torch.repeat_interleave(torch.arange(s["b"], device="cuda"), count, output_size=s["touched"])
        j = first[seq] + torch.arange(s["touched"], device="cuda") - (count.cumsum(0) - count)[seq]
        ids = s["block_tables"][seq, j].long()
        seen = torch.arange(bs, device="cuda")[None, :] + j[:, None] * bs < s["lens"][seq][:, None]
        k = _values(s["k_cache"][ids], s) if not s["fp8"] else _values(s["k_cache"], s)[ids]
        hi = k.masked_fill(~seen[:, None, :, None], float("-inf")).amax(2)
        lo = k.masked_fill(~seen[:, None, :, None], float("inf")).amin(2)
        step = _step(torch.maximum(hi.abs(), lo.abs()).amax(-1))
        codes[ids] = _codes(torch.stack([hi, lo], 2), step[..., None, None]).to(torch.int8)
        steps[ids] = step
    return codes * steps[:, :, None, None]


def _run_select(s):
    if own:
        return s["pool"].select_blocks(s["q"], s["bounds"], s["block_tables"], s["lens"], s["budget"], s["first"], s["last"])
    b, bs, hkv, d, budget = s["b"], s["bs"], s["hkv"], s["d"], s["budget"]
    grp, tables = s["hq"] // hkv, s["block_tables"].long()
    codes, steps = _bounds_of(s)
    q = s["q"].float().view(b, s["q_len"], hkv, grp, d).transpose(1, 2).reshape(b, hkv, -1, d)
    q_step = _step(q.abs().amax(-1))
    c = _codes(q, q_step[..., None])
    n = tables.shape[1]
    # sum of max(c hi, c lo): the upper bound where c is positive, the lower one where it is negative
    hi, lo = (codes[:, :, i][tables].float().permute(0, 2, 3, 1) for i in (0, 1))
    dot = torch.matmul(c.clamp(min=0), hi) + torch.matmul(c.clamp(max=0), lo)
    score = (dot * q_step[..., None]).amax(2) * steps[tables].transpose(1, 2)
    count = ((s["lens"] + bs - 1) // bs)[:, None, None]
    at = torch.arange(n, device="cuda")
    score = torch.where((at < s["first"]) | (at >= count - s["last"]), float("inf"), score)
    score = score.masked_fill(at >= count, float("-inf"))
    # a stable order keeps the lowest index of equal scores in front
    pick = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :budget]
    pick = torch.where(pick < count, pick, 2 ** 30).sort(-1).values
    pick = torch.where(pick < 2 ** 30, pick, -1).to(torch.int32)
    return torch.nn.functional.pad(pick, (0, budget - pick.shape[-1]), value=-1)


def _run_attend(s):
    if own:
        return s["pool"].decode_selected(s["q"], s["selected"], s["block_tables"], s["lens"], s["scale"])
    b, n, bs, hkv, d, budget = s["b"], s["q_len"], s["bs"], s["hkv"], s["d"], s["budget"]
    grp, keys = s["hq"] // hkv, budget * bs
    chosen = s["selected"].clamp(min=0).long()
    ids = s["block_tables"].long().gather(1, chosen.view(b, -1)).view(b, hkv, budget)
    head = torch.arange(hkv, device="cuda")[None, :, None]
    if s["fp8"]:
        k, v = (_values(x, s)[ids, head].view(b, hkv, keys, d) for x in (s["k_cache"], s["v_cache"]))
    else:
        k, v = (x[ids, head].float().view(b, hkv, keys, d) for x in (s["k_cache"], s["v_cache"]))
    off = torch.arange(bs, device="cuda")
    pos = (chosen[..., None] * bs + off).masked_fill(s["selected"][..., None] < 0, 2 ** 30).view(b, hkv, 1, 1, keys)
    last = s["lens"][:, None] - n + torch.arange(n, device="cuda")
    q = s["q"].float().view(b, n, hkv, grp, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, n * grp, d)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(b, hkv, n, grp, keys)
    x = x.masked_fill(pos > last[:, None, :, None, None], float("-inf"))
    x = (x - x.amax(-1, keepdim=True).clamp_(min=-1e30)).exp_()
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x.view(b, hkv, n * grp, keys), v).view(b, hkv, n, grp, d) / torch.where(total > 0, total, 1.0)
    return out.permute(0, 2, 1, 3, 4).reshape(b, n, s["hq"], d).to(s["q"].dtype)


# -------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": _exact_tables, "bounds": _exact_bounds, "select": _exact_select, "attend": _exact_attend}[s["op"]](s)


def _exact_tables(s):
    """A step on the host, one sequence after the other."""
    bs, rows = s["bs"], s["block_tables"].tolist()
    store, free = s["free"].tolist(), int(s["num_free"])
    lens, new = s["lens"].tolist(), s["new"].tolist()
    kept = [min(n, k) for n, k in zip(lens, s["keep"].tolist())]
    back = [row[_blocks(k, bs):_blocks(n, bs)] for row, n, k in zip(rows, lens, kept)]
    for row in reversed(back):
        for i in reversed(row):
            store[free] = i
            free += 1
    cu, positions, slots = [0], [], []
    for i, row in enumerate(rows):
        for j in range(_blocks(kept[i], bs), _blocks(kept[i] + new[i], bs)):
            free -= 1
            row[j] = store[free]
        for p in range(kept[i], kept[i] + new[i]):
            positions.append(p)
            slots.append(row[p // bs] * bs + p % bs)
        cu.append(len(slots))
    behind = s["num_tokens"] - len(slots)
    return (_i32(rows), _i32([k + n for k, n in zip(kept, new)]), _i32(store), _i32([free]), _i32(cu),
            _i32(positions + [0] * behind), torch.tensor(slots + [-1] * behind, dtype=torch.int64, device="cuda"))


def _exact_bounds(s):
    bs, hkv, d = s["bs"], s["hkv"], s["d"]
    codes, steps = _bounds_of(s)
    out = codes.double() * steps.double()[:, :, None, None]
    size = s["nb"] * hkv * bs * d
    cu, lens, tables = s["cu_q"].tolist(), s["lens"].tolist(), s["block_tables"].tolist()
    if s["fp8"]:
        # an 8-bit pool's keys are numbers of 32 bits: code * scale, rounded
        scale = s["k_cache"][size:].view(torch.float32)
        keys = s["k_cache"][:size].view(torch.float8_e4m3fn).float().view(-1, d).mul(scale[:, None]).double()
        keys = keys.view(s["nb"], hkv, bs, d)
    for i, n in enumerate(lens):
        first, full = (n - (cu[i + 1] - cu[i])) // bs, n // bs
        for lo, hi, rows in ((first, full, bs), (full, full + (n % bs > 0), n % bs)):
            if lo >= hi:
                continue
            ids = torch.tensor(tables[i][lo:hi], device="cuda")
            k = (keys[ids] if s["fp8"] else s["k_cache"][ids].double())[:, :, :rows]
            both = torch.stack([k.max(2).values, k.min(2).values], 2)
            top = both.abs().amax((2, 3), keepdim=True)
            step = torch.exp2(torch.ceil(torch.log2(top / 127.0)))
            out[ids] = torch.round(both / step) * step
    return out


def _exact_select(s):
    import numpy as np
    b, bs, hkv, d, budget = s["b"], s["bs"], s["hkv"], s["d"], s["budget"]
    grp = s["hq"] // hkv
    codes, steps = (x.cpu().numpy().astype(np.float64) for x in _bounds_of(s))
    tables, lens = s["block_tables"].cpu().numpy(), s["lens"].tolist()
    q = s["q"].double().cpu().numpy()
    out = np.full((b, hkv, budget), -1, dtype=np.int32)
    for i in range(b):
        n = _blocks(lens[i], bs)
        if n * hkv * s["hq"] * s["q_len"] * d > 2 ** 33:
            return None
        for h in range(hkv):
            k = codes[tables[i, :n], h]
            best = np.full(n, -np.inf)
            for row in q[i, :, h * grp:(h + 1) * grp].reshape(-1, d):
                step = 2.0 ** np.ceil(np.log2(np.abs(row).max() / 127.0))
                c = np.rint(row / step)
                side = np.where(c > 0, k[:, 0], k[:, 1])
                best = np.maximum(best, side @ c * step * steps[tables[i, :n], h])
            best[:s["first"]] = np.inf
            best[max(0, n - s["last"]):] = np.inf
            pick = np.sort(np.lexsort((np.arange(n), -best))[:budget])
            out[i, h, :len(pick)] = pick
    return torch.from_numpy(out).cuda()


def _exact_attend(s):
    n, bs, hkv, d = s["q_len"], s["bs"], s["hkv"], s["d"]
    grp, size = s["hq"] // hkv, s["nb"] * hkv * bs * d
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lens, selected = s["lens"].tolist(), s["selected"].tolist()

    def rows(cache, ids, h):
        if not s["fp8"]:
            return cache[ids, h].double().reshape(-1, d)
        codes = cache[:size].view(torch.float8_e4m3fn).view(s["nb"], hkv, bs, d)[ids, h].double()
        scale = cache[size:].view(torch.float32).view(s["nb"], hkv, bs)[ids, h].double()
        return (codes * scale[..., None]).reshape(-1, d)

    for i in range(s["b"]):
        for h in range(hkv):
            chosen = torch.tensor([j for j in selected[i][h] if j >= 0], dtype=torch.int64, device="cuda")
            ids = s["block_tables"][i].long()[chosen]
            pos = (chosen[:, None] * bs + torch.arange(bs, device="cuda")).reshape(-1)
            k, v = rows(s["k_cache"], ids, h), rows(s["v_cache"], ids, h)
            heads = slice(h * grp, (h + 1) * grp)
            for r in range(n):
                seen = (pos <= lens[i] - n + r).nonzero()[:, 0]
                if seen.numel():
                    x = s["q"][i, r, heads].double() @ k[seen].T * s["scale"]
                    out[i, r, heads] = torch.softmax(x, -1) @ v[seen]
    return out
