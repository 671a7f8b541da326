"""Definitions of step_tables, key_bounds, select_blocks and decode_selected (Python and numpy on the host, 64 bits)."""
import math

import numpy as np
import torch


def ceil_div(a, b):
    return -(-a // b)


def step_tables(new, lens, rows, free, num_free, num_tokens, bs, keep=None):
    """One sequence after the other. rows: lists; free: a list of num_blocks ids. Returns everything anew."""
    rows, free = [list(r) for r in rows], list(free)
    kept = [min(n, k) for n, k in zip(lens, keep)] if keep is not None else list(lens)
    for row, n, k in reversed(list(zip(rows, lens, kept))):
        for i in reversed(row[ceil_div(k, bs):ceil_div(n, bs)]):
            free[num_free] = i
            num_free += 1
    cu, pos, slots = [0], [], []
    for row, k, m in zip(rows, kept, new):
        for j in range(ceil_div(k, bs), ceil_div(k + m, bs)):
            num_free -= 1
            row[j] = free[num_free]
        pos += range(k, k + m)
        slots += [row[p // bs] * bs + p % bs for p in range(k, k + m)]
        cu.append(len(slots))
    pad = num_tokens - len(slots)
    return rows, [k + m for k, m in zip(kept, new)], free, num_free, cu, pos + [0] * pad, slots + [-1] * pad


def step_of(top):
    """The smallest power of two s (of fp32's numbers) with top <= 127 s; 0 for 0, infinity for what is no number."""
    if not top < math.inf:
        return math.inf
    if top == 0:
        return 0.0
    m, e = math.frexp(top)
    return max(math.ldexp(1.0, e - 7 + (m > 127 / 128)), 2.0 ** -149)


def bounds_of(keys):
    """keys [n, d] (numpy float64) -> codes [2, d] (int), step."""
    hi, lo = keys.max(0), keys.min(0)                   # NaN is kept
    top = np.max(np.abs(np.stack([hi, lo])))
    step = step_of(float(top))
    if step == math.inf or step == 0:
        return np.zeros((2, keys.shape[1]), int), step
    return np.rint(np.stack([hi, lo]) / step).astype(int), step


def select(q, codes, steps, row, length, bs, budget, first, last):
    """One (sequence, KV head): q [rows, d] float64, codes [nb, 2, d], steps [nb], row: the table's ids."""
    n = ceil_div(length, bs)
    out = np.full(budget, -1)
    if n <= budget:
        out[:n] = np.arange(n)
        return out
    known = (row[:n] >= 0) & (row[:n] < len(codes))
    ids = np.where(known, row[:n], 0)
    c = codes[ids].astype(np.float64)
    s = steps[ids]
    best = np.full(n, -np.inf)
    for x in q:
        step = step_of(float(np.abs(x).max()) if np.isfinite(x).all() else math.inf)
        if step == math.inf:
            continue
        k = np.rint(x / step) if step else np.zeros_like(x)
        dot = np.maximum(k * c[:, 0], k * c[:, 1]).sum(1)
        with np.errstate(invalid="ignore"):
            best = np.maximum(best, dot * step)
    with np.errstate(invalid="ignore"):
        score = np.where(np.isinf(s), np.inf, np.where(s == 0, 0.0, best * s))
    score = np.where(known, score, -np.inf)              # an id outside the pool
    forced = (np.arange(n) < first) | (np.arange(n) >= n - last)
    pick = np.lexsort((np.arange(n), -score, ~forced))[:budget]
    out[:] = np.sort(pick)
    return out


def attend(q, keys, values, selected, lens, scale):
    """q [B, n, Hq, d]; keys, values: functions (b, h, j) -> the block's rows [bs, d] in float64; selected [B, Hkv, S].
    Returns out, the sums of weights times |values|, and for each row the largest sum of |q k| scale (all float64)."""
    B, n, hq, d = q.shape
    hkv = selected.shape[1]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    mag, big = torch.zeros_like(out), torch.zeros(B, n, hq, dtype=torch.float64, device=q.device)
    for b in range(B):
        for h in range(hkv):
            js = [j for j in selected[b][h].tolist() if j >= 0]
            if not js:
                continue
            k = torch.cat([keys(b, h, j) for j in js])
            v = torch.cat([values(b, h, j) for j in js])
            bs = k.shape[0] // len(js)
            pos = torch.cat([torch.arange(j * bs, (j + 1) * bs, device=q.device) for j in js])
            G = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            for r in range(n):
                seen = (pos <= int(lens[b]) - n + r).nonzero()[:, 0]
                if not seen.numel():
                    continue
                x = q[b, r, G].double()
                p = torch.softmax(x @ k[seen].T * scale, -1)
                out[b, r, G] = p @ v[seen]
                mag[b, r, G] = p @ v[seen].abs()
                big[b, r, G] = (x.abs() @ k[seen].abs().T).amax(-1) * abs(scale)
    return out, mag, big
