"""Measured cases of three serving operators: rope_append, prefill_packed and the token-distribution
pair adjust_logits / token_probs.

With `own` false, run() computes each operator in its plain form (elementary torch operations in 32
bits, angles in 64); with `own` true it calls the library. prepare() makes the inputs from the seed
and what a serving program keeps: the KV pool's handle and the rotation's frequency table.
"""
import math
import random

import torch

own = False

_DTYPE = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # rope_append: one new token of one sequence, the shortest call of a decode loop
        dict(name="rope-1", op="rope", n=1, hq=32, hkv=8, d=128, dtype="bf16", fp8=False, bs=16, rot=128,
             interleaved=False, fused=False, maxpos=2000, spare=64),
        # rope_append: a decode step of a large batch at far positions
        dict(name="rope-decode-256", op="rope", n=256, hq=64, hkv=8, d=128, dtype="fp16", fp8=False, bs=16, rot=128,
             interleaved=False, fused=True, maxpos=131072, spare=256),
        # rope_append: a step of prompt tokens, q, k and v as slices of one fused projection's output
        dict(name="rope-prompt-8192", op="rope", n=8192, hq=64, hkv=8, d=128, dtype="bf16", fp8=False, bs=16, rot=128,
             interleaved=False, fused=True, maxpos=8192, spare=0),
        # rope_append: an odd number of tokens into an FP8 pool, neighbouring pairs, half of the dimensions rotated
        dict(name="rope-fp8-2049", op="rope", n=2049, hq=32, hkv=8, d=128, dtype="bf16", fp8=True, bs=32, rot=64,
             interleaved=True, fused=True, maxpos=40000, spare=31),
        # prefill_packed: one short prompt, where latency counts
        dict(name="prompt-77", op="prompt", b=1, new_lo=77, new_hi=77, old_lo=0, old_hi=0, mix=1, hq=32, hkv=8, d=128,
             dtype="bf16", bs=16),
        # prefill_packed: prompts of very different lengths, one token among them, as they arrive together
        dict(name="prompt-mixed-32", op="prompt", b=32, new_lo=1, new_hi=2000, old_lo=0, old_hi=0, mix=2, hq=32,
             hkv=8, d=128, dtype="bf16", bs=16),
        # prefill_packed: long whole prompts, many heads: the largest call
        dict(name="prompt-4x4096", op="prompt", b=4, new_lo=4096, new_hi=4096, old_lo=0, old_hi=0, mix=3, hq=64,
             hkv=8, d=128, dtype="bf16", bs=16),
        # prefill_packed: few new tokens behind long cached contexts (a prefix found in the cache, a next turn)
        dict(name="prompt-cached-3", op="prompt", b=3, new_lo=5, new_hi=64, old_lo=20000, old_hi=65536, mix=4, hq=32,
             hkv=8, d=128, dtype="fp16", bs=32),
        # prefill_packed: small heads, one KV head per query head
        dict(name="prompt-d64", op="prompt", b=5, new_lo=300, new_hi=2048, old_lo=0, old_hi=500, mix=5, hq=16,
             hkv=16, d=64, dtype="fp16", bs=16),
        # token_probs: one sequence's next-token distribution
        dict(name="probs-1", op="logits", b=1, r=1, v=32000, pad=0, dtype="fp32", hist=200, nbias=8, mask=False,
             draft=False, probs=True),
        # adjust_logits: a decode step's logits, 16-bit, handed on to the caller's own sampler
        dict(name="logits-64", op="logits", b=64, r=1, v=128256, pad=0, dtype="bf16", hist=2048, nbias=300, mask=True,
             draft=False, probs=False),
        # token_probs: the target's distributions for a verify of five drafts per sequence, with a grammar's masks
        dict(name="probs-verify-64x6", op="logits", b=64, r=6, v=128256, pad=0, dtype="fp32", hist=4096, nbias=32,
             mask=True, draft=True, probs=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "prompt", "prompt", "logits"])
    if op == "rope":
        d = rng.choice([64, 128, 128])
        hq, hkv = rng.choice([(32, 8), (64, 8), (16, 16), (8, 1), (20, 4), (12, 4)])
        fp8 = d == 128 and rng.random() < 0.3
        return dict(op="rope", n=_log(rng, 1, 8192), hq=hq, hkv=hkv, d=d, dtype=rng.choice(["bf16", "fp16"]), fp8=fp8,
                    bs=rng.choice([16, 32]), rot=rng.choice([d, d, d // 2, 32]), interleaved=rng.random() < 0.5,
                    fused=rng.random() < 0.5, maxpos=_log(rng, 100, 1000000), spare=rng.randrange(0, 300))
    if op == "prompt":
        while True:
            hq, hkv = rng.choice([(32, 8), (64, 8), (16, 16), (8, 1), (20, 4), (12, 4)])
            new_hi = _log(rng, 1, 4096)
            old_hi = rng.choice([0, 0, _log(rng, 16, 65536)])
            c = dict(op="prompt", b=_log(rng, 1, 32), new_lo=rng.choice([1, new_hi, max(1, new_hi // 4)]),
                     new_hi=new_hi, old_lo=old_hi // rng.choice([1, 2, 8]), old_hi=old_hi,
                     mix=rng.randrange(1, 1000000), hq=hq, hkv=hkv, d=rng.choice([64, 128, 128]),
                     dtype=rng.choice(["bf16", "fp16"]), bs=rng.choice([16, 32]))
            longest = c["new_hi"] + c["old_hi"] + c["bs"]
            if (c["b"] * hq * c["new_hi"] * longest <= 2 ** 31 and c["b"] * longest * hkv * c["d"] <= 3 * 10 ** 8):
                return c
    while True:
        r = rng.choice([1, 1, 2, 4, 6])
        c = dict(op="logits", b=_log(rng, 1, 64), r=r, v=_log(rng, 1000, 262144), pad=rng.choice([0, 0, 1, 64]),
                 dtype=rng.choice(["fp32", "bf16", "fp16"]), hist=rng.choice([0, _log(rng, 1, 4096)]),
                 nbias=rng.choice([0, 1, 300]), mask=rng.random() < 0.5, draft=r > 1, probs=rng.random() < 0.7)
        if c["b"] * r * c["v"] <= 64 * 6 * 128256 // 2:
            return c


def _lens(case):
    """New and cached tokens of each sequence: spread over the logarithm, fixed by the case."""
    rng = random.Random(case["mix"])
    new = [_log(rng, case["new_lo"], case["new_hi"]) for _ in range(case["b"])]
    old = [_log(rng, case["old_lo"], case["old_hi"]) if case["old_lo"] > 0 else
           (rng.randint(0, case["old_hi"]) if case["old_hi"] else 0) for _ in range(case["b"])]
    return new, old


def work(case):
    if case["op"] == "rope":
        n, d = case["n"], case["d"]
        rows = n * (case["hq"] + 2 * case["hkv"]) * d * 2
        kv_out = 2 * n * case["hkv"] * ((d + 4) if case["fp8"] else 2 * d)
        pairs = n * (case["hq"] + case["hkv"]) * case["rot"] // 2
        return {"bytes": rows + n * case["hq"] * d * 2 + kv_out + n * 12, "flops": 6 * pairs}
    if case["op"] == "prompt":
        new, old = _lens(case)
        pairs = sum(o * n + n * (n + 1) // 2 for n, o in zip(new, old))
        rows, keys = sum(new), sum(new) + sum(old)
        return {"bytes": 2 * case["d"] * (2 * rows * case["hq"] + 2 * keys * case["hkv"]),
                "flops": 4 * case["d"] * case["hq"] * pairs}
    rows, v = case["b"] * case["r"], case["v"]
    size = 4 if case["dtype"] == "fp32" else 2
    return {"bytes": rows * v * (size + 4) + (rows * ((v + 31) // 32) * 4 if case["mask"] else 0) +
            case["b"] * (case["hist"] * 4 + case["nbias"] * 8), "flops": rows * v * (8 if case["probs"] else 4)}


# ----------------------------------------------------------------------------------- the inputs

def _inv_freq(rot):
    """Frequencies of the rotation, as a model's configuration gives them (base 500000)."""
    return [500000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DTYPE[case["dtype"]]
    s = dict(case)
    return {"rope": _prepare_rope, "prompt": _prepare_prompt, "logits": _prepare_logits}[case["op"]](s, g, dt)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _prepare_rope(s, g, dt):
    n, hq, hkv, d, bs = s["n"], s["hq"], s["hkv"], s["d"], s["bs"]
    qkv = torch.empty(n, (hq + 2 * hkv) * d, dtype=dt, device="cuda").copy_(_randn(g, n, (hq + 2 * hkv) * d))
    q, k, v = qkv.split([hq * d, hkv * d, hkv * d], dim=1)
    q, k, v = q.view(n, hq, d), k.view(n, hkv, d), v.view(n, hkv, d)
    s["q"], s["k"], s["v"] = (q, k, v) if s["fused"] else (q.contiguous(), k.contiguous(), v.contiguous())
    s["positions"] = torch.randint(0, s["maxpos"], (n,), generator=g, device="cuda", dtype=torch.int32)
    nb = (n + s["spare"] + bs - 1) // bs
    s["slots"] = torch.randperm(nb * bs, generator=g, device="cuda")[:n].contiguous()
    s["nb"] = nb
    if s["fp8"]:
        size = nb * hkv * bs
        for name in ("k_cache", "v_cache"):
            codes = _randn(g, size * d).to(torch.float8_e4m3fn).view(torch.uint8)
            scales = torch.rand(size, generator=g, device="cuda") * 0.01 + 0.001
            s[name] = torch.cat([codes, scales.view(torch.uint8)])
    else:
        for name in ("k_cache", "v_cache"):
            s[name] = _randn(g, nb, hkv, bs, d).to(dt)
    s["inv_freq"] = torch.tensor(_inv_freq(s["rot"]), dtype=torch.float64, device="cuda")
    if own:
        from paged_kv_cache_223_gb300 import pagedattn as pa
        s["rope"] = pa.Rope(_inv_freq(s["rot"]), interleaved=s["interleaved"])
        s["pool"] = pa.Pool(nb, bs, hkv, d, dtype=dt, max_seqs=1, max_context_len=512, k_cache=s["k_cache"],
                            v_cache=s["v_cache"], kv_format=pa.PA_KV_FP8_E4M3 if s["fp8"] else pa.PA_KV_16BIT)
    return s


def _prepare_prompt(s, g, dt):
    new, old = _lens(s)
    b, hq, hkv, d, bs = s["b"], s["hq"], s["hkv"], s["d"], s["bs"]
    lens = [x + y for x, y in zip(new, old)]
    blocks = [(x + bs - 1) // bs for x in lens]
    nb, stride = sum(blocks), max(blocks)
    s["q"] = (_randn(g, sum(new), hq, d) * 1.5).to(dt)
    s["k_cache"] = _randn(g, nb, hkv, bs, d).to(dt)
    s["v_cache"] = (_randn(g, nb, hkv, bs, d) + 0.5 * _randn(g, 1, hkv, 1, d)).to(dt)
    ids = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    tables = torch.zeros(b, stride, dtype=torch.int32, device="cuda")
    at = 0
    for i, m in enumerate(blocks):
        tables[i, :m] = ids[at:at + m]
        at += m
    s["tables"] = tables
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    s["cu_q"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["scale"] = 1.0 / math.sqrt(d)
    s["longest_new"] = max(new)
    if own:
        from paged_kv_cache_223_gb300 import pagedattn as pa
        s["pool"] = pa.Pool(nb, bs, hkv, d, dtype=dt, max_seqs=b, max_q_heads=hq, max_q_len=1,
                            max_context_len=max(lens), k_cache=s["k_cache"], v_cache=s["v_cache"])
    return s


def _prepare_logits(s, g, dt):
    b, r, v = s["b"], s["r"], s["v"]
    full = (_randn(g, b, r, v + s["pad"]) * 3.0).to(dt)
    s["logits"] = full[:, :, :v]
    # token ids as text has them: a few frequent ones, many rare ones
    ids = lambda *shape: (torch.rand(shape, generator=g, device="cuda").pow(3) * v).to(torch.int32).clamp_(max=v - 1)  # noqa: E731
    h = s["hist"]
    s["history"] = ids(b, h)
    s["history_lens"] = torch.randint(0, h + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
    s["prompt_lens"] = (s["history_lens"] * torch.rand(b, generator=g, device="cuda")).to(torch.int32)
    s["draft"] = ids(b, r - 1) if s["draft"] else None
    rand = lambda lo, hi: torch.rand(b, generator=g, device="cuda") * (hi - lo) + lo  # noqa: E731
    s["repetition"], s["presence"], s["frequency"] = rand(1.0, 1.3), rand(0.0, 1.0), rand(0.0, 0.5)
    # per-request biases: the rows' lists are filled up with -1
    s["bias_tokens"] = ids(b, s["nbias"])
    keep = torch.randint(0, s["nbias"] + 1, (b, 1), generator=g, device="cuda")
    s["bias_tokens"][torch.arange(s["nbias"], device="cuda")[None, :] >= keep] = -1
    s["bias_values"] = _randn(g, b, s["nbias"]) * 2.0
    words = (v + 31) // 32
    s["mask_words"] = torch.randint(-2 ** 31, 2 ** 31, (b, r, words), generator=g, device="cuda",
                                    dtype=torch.int64).to(torch.int32) if s["mask"] else None
    s["temperature"] = rand(0.5, 1.2)
    s["temperature"][::7] = torch.where(torch.arange(0, b, 7, device="cuda") > 0, 0.0, s["temperature"][::7])
    return s


# ------------------------------------------------------------------------------------ one pass

def run(s):
    return {"rope": _run_rope, "prompt": _run_prompt, "logits": _run_logits}[s["op"]](s)


def _dequantised(cache, s, dt):
    """An FP8 cache's values: code * scale, in the pool's model type."""
    rows = s["nb"] * s["hkv"] * s["bs"]
    codes = cache[:rows * s["d"]].view(torch.float8_e4m3fn).float().view(rows, s["d"])
    return (codes * cache[rows * s["d"]:].view(torch.float32)[:, None]).to(dt)


def _rotated(x, cos, sin, s):
    """x [n, h, d] in 32 bits with its first `rot` dimensions rotated, pair i by angle i."""
    rot = s["rot"]
    c, t = cos[:, None, :], sin[:, None, :]
    y = x.clone()
    if s["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * t, b * c + a * t
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * t, b * c + a * t
    return y


def _run_rope(s):
    dt = _DTYPE[s["dtype"]]
    if own:
        q = s["pool"].rope_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["rope"])
    else:
        angle = s["positions"].double()[:, None] * s["inv_freq"][None, :]
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
        q = _rotated(s["q"].float(), cos, sin, s).to(dt)
        k = _rotated(s["k"].float(), cos, sin, s)
        blk, off = s["slots"] // s["bs"], s["slots"] % s["bs"]
        if s["fp8"]:
            rows = s["nb"] * s["hkv"] * s["bs"]
            at = (blk[:, None] * s["hkv"] + torch.arange(s["hkv"], device="cuda")[None, :]) * s["bs"] + off[:, None]
            for cache, x in ((s["k_cache"], k), (s["v_cache"], s["v"].float())):
                amax = x.abs().amax(-1)
                scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
                codes = (x / scale[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
                cache[:rows * s["d"]].view(rows, s["d"])[at] = codes
                cache[rows * s["d"]:].view(torch.float32)[at] = scale
        else:
            s["k_cache"][blk, :, off] = k.to(dt)
            s["v_cache"][blk, :, off] = s["v"]
    if s["fp8"]:
        return q, _dequantised(s["k_cache"], s, dt), _dequantised(s["v_cache"], s, dt)
    return q, s["k_cache"], s["v_cache"]


def _run_prompt(s):
    if own:
        return s["pool"].prefill_packed(s["q"], s["cu_q"], s["tables"], s["lens"], s["scale"])
    b, hq, hkv, d, n = s["b"], s["hq"], s["hkv"], s["d"], s["longest_new"]
    total, grp = s["q"].shape[0], hq // hkv
    tok = torch.arange(total, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["cu_q"][1:], tok, right=True)
    row = tok - s["cu_q"][seq]
    q = torch.zeros(b, n, hq, d, device="cuda")
    q[seq, row] = s["q"].float()
    q = q.view(b, n, hkv, grp, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, grp * n, d)
    tables = s["tables"].long()
    keys = tables.shape[1] * s["bs"]
    k = s["k_cache"][tables].float().permute(0, 2, 1, 3, 4).reshape(b, hkv, keys, d)
    v = s["v_cache"][tables].float().permute(0, 2, 1, 3, 4).reshape(b, hkv, keys, d)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(b, hkv, grp, n, keys)
    first = s["lens"] - (s["cu_q"][1:] - s["cu_q"][:-1])
    last = first[:, None] + torch.arange(n, device="cuda")[None, :]
    hidden = torch.arange(keys, device="cuda")[None, None, :] > last[:, :, None]
    x.masked_fill_(hidden[:, None, None], float("-inf"))
    x.sub_(x.amax(-1, keepdim=True)).exp_()
    weight = x.sum(-1, keepdim=True)
    out = torch.matmul(x.view(b, hkv, grp * n, keys), v).view(b, hkv, grp, n, d) / weight
    return out.permute(0, 3, 1, 2, 4).reshape(b, n, hq, d)[seq, row].to(s["q"].dtype)


def _run_logits(s):
    if own:
        from paged_kv_cache_223_gb300 import pagedattn as pa
        kw = dict(history=s["history"], history_lens=s["history_lens"], prompt_lens=s["prompt_lens"],
                  draft=s["draft"], repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
                  bias_tokens=s["bias_tokens"], bias_values=s["bias_values"], mask=s["mask_words"])
        return pa.token_probs(s["logits"], s["temperature"], **kw) if s["probs"] else pa.adjust_logits(s["logits"], **kw)
    b, r, v, h, nb = s["b"], s["r"], s["v"], s["hist"], s["nbias"]
    x = s["logits"].float()
    at = torch.arange(h, device="cuda", dtype=torch.int32)[None, :]
    known = (at < s["history_lens"][:, None]).float()
    made = known * (at >= s["prompt_lens"][:, None])
    tokens = s["history"].long()
    seen = torch.zeros(b, 1, v, device="cuda")
    count = torch.zeros(b, r, v, device="cuda")
    seen[:, 0].scatter_add_(1, tokens, known)
    count[:, 0].scatter_add_(1, tokens, made)
    if s["draft"] is not None:
        count[:, 1:].scatter_(2, s["draft"].long()[:, :, None], 1.0)
    count = count.cumsum(1) if r > 1 else count
    rep = s["repetition"][:, None, None]
    x = torch.where((seen + count) > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = x - s["frequency"][:, None, None] * count
    x = x - s["presence"][:, None, None] * (count > 0)
    # the last entry that names a token counts
    order = torch.arange(1, nb + 1, device="cuda")[None, :].expand(b, nb)
    order = torch.where(s["bias_tokens"] >= 0, order, torch.zeros_like(order))
    last = torch.zeros(b, v, dtype=torch.int64, device="cuda")
    last.scatter_reduce_(1, s["bias_tokens"].long().clamp(min=0), order, "amax")
    values = torch.cat([torch.zeros(b, 1, device="cuda"), s["bias_values"]], dim=1)
    x = x + values.gather(1, last)[:, None, :]
    if s["mask_words"] is not None:
        bit = torch.arange(v, device="cuda")
        allowed = (s["mask_words"][:, :, bit // 32] >> (bit % 32).to(torch.int32)) & 1
        x = x.masked_fill(allowed == 0, float("-inf"))
    if not s["probs"]:
        return x
    t = s["temperature"][:, None, None]
    top = x.amax(-1, keepdim=True)
    best = torch.where(x == top, torch.arange(v, device="cuda"), v).amin(-1, keepdim=True)
    greedy = (torch.arange(v, device="cuda") == best).float()
    e = torch.exp((x - top) / torch.where(t > 0, t, torch.ones_like(t)))
    return torch.where(t > 0, e / e.sum(-1, keepdim=True), greedy)


# -------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "prompt": _exact_prompt, "logits": _exact_logits}[case["op"]](s)


def _exact_rope(s):
    rot, d, hkv, bs = s["rot"], s["d"], s["hkv"], s["bs"]
    freq = torch.tensor(_inv_freq(rot), dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.ones_like(freq)[None, :].expand(s["n"], -1).contiguous(),
                       s["positions"].double()[:, None] * freq)

    def turned(x):
        x = x.double()
        head, rest = x[..., :rot], x[..., rot:]
        if s["interleaved"]:
            z = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous()) * turn[:, None, :]
            return torch.cat([torch.view_as_real(z).reshape(head.shape), rest], dim=-1)
        z = torch.complex(head[..., :rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * turn[:, None, :]
        return torch.cat([z.real, z.imag, rest], dim=-1)

    q, k, v = turned(s["q"]), turned(s["k"]), s["v"].double()
    caches = []
    for name, x in (("k_cache", k), ("v_cache", v)):
        rows = s["nb"] * hkv * bs
        if s["fp8"]:
            codes = s[name][:rows * d].view(torch.float8_e4m3fn).double().view(rows, d)
            whole = codes * s[name][rows * d:].view(torch.float32).double()[:, None]
            top = x.abs().amax(-1, keepdim=True) / 448.0
            step = torch.where(top > 0, top, torch.ones_like(top))
            # E4M3: three bits behind the leading one, down to 2^-6; below it steps of 2^-9
            y = x / step
            grain = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            x = torch.round(y / grain) * grain * step
        else:
            whole = s[name].double().reshape(rows, d)
        head = torch.arange(hkv, device="cuda")
        for_row = ((s["slots"] // bs)[:, None] * hkv + head) * bs + (s["slots"] % bs)[:, None]
        whole[for_row.reshape(-1)] = x.reshape(-1, d)
        caches.append(whole if s["fp8"] else whole.view(s["nb"], hkv, bs, d))
    return q, caches[0], caches[1]


def _exact_prompt(s):
    new, old = _lens(s)
    hq, hkv, d, bs = s["hq"], s["hkv"], s["d"], s["bs"]
    out, at = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), 0
    for i, (n, o) in enumerate(zip(new, old)):
        ids = s["tables"][i, :(n + o + bs - 1) // bs].long()
        for h in range(hkv):
            k = s["k_cache"][ids, h].reshape(-1, d)[:n + o].double()
            v = s["v_cache"][ids, h].reshape(-1, d)[:n + o].double()
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            x = torch.einsum("nhd,td->hnt", s["q"][at:at + n, heads].double(), k) * s["scale"]
            seen = torch.ones(n, n + o, dtype=torch.bool, device="cuda").tril(o)
            p = torch.softmax(torch.where(seen, x, float("-inf")), dim=-1)
            out[at:at + n, heads] = torch.einsum("hnt,td->nhd", p, v)
        at += n
    return out


def _exact_logits(s):
    b, r, v = s["b"], s["r"], s["v"]
    out = torch.empty(b, r, v, dtype=torch.float64, device="cuda")
    bit = torch.arange(v, device="cuda")
    for i in range(b):
        n, m = int(s["history_lens"][i]), int(s["prompt_lens"][i])
        past = s["history"][i, :n].long()
        bias = torch.zeros(v, dtype=torch.float64, device="cuda")
        entries = dict(zip(s["bias_tokens"][i].tolist(), s["bias_values"][i].tolist()))
        entries.pop(-1, None)
        if entries:
            bias[torch.tensor(list(entries), device="cuda")] = torch.tensor(list(entries.values()),
                                                                            dtype=torch.float64, device="cuda")
        rep, pres, freq, t = (float(s[k][i]) for k in ("repetition", "presence", "frequency", "temperature"))
        for j in range(r):
            x = s["logits"][i, j].double()
            made = past[m:] if s["draft"] is None else torch.cat([past[m:], s["draft"][i, :j].long()])
            count = torch.bincount(made, minlength=v)
            seen = (torch.bincount(past, minlength=v) + count) > 0
            x = torch.where(seen & (x > 0), x / rep, torch.where(seen, x * rep, x))
            x = x - freq * count - pres * (count > 0) + bias
            if s["mask_words"] is not None:
                words = s["mask_words"][i, j].long() & 0xFFFFFFFF
                x = torch.where(((words[bit >> 5] >> (bit & 31)) & 1) > 0, x, float("-inf"))
            if not s["probs"]:
                out[i, j] = x
            elif t > 0:
                out[i, j] = torch.softmax(x / t, dim=-1)
            else:
                out[i, j] = 0.0
                out[i, j, (x == x.max()).nonzero()[0, 0]] = 1.0
    return out
