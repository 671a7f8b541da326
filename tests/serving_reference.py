"""Definitions of rope_append, prefill_packed, adjust_logits and token_probs in 64 bits (torch, any device)."""
import math

import torch


def rotate(x, positions, inv_freq, interleaved, scale=1.0):
    """x [N, H, d] -> float64, its first 2 * len(inv_freq) dimensions turned; and sum of |terms| per element."""
    x = x.double()
    f = torch.as_tensor(inv_freq, dtype=torch.float64, device=x.device)
    rot = 2 * f.numel()
    ang = (positions.double()[:, None] * f[None, :])[:, None, :]
    c, s = torch.cos(ang) * scale, torch.sin(ang) * scale
    y, mag = x.clone(), x.abs()
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + (1 if interleaved else rot // 2)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = (a.abs() + b.abs()) * abs(scale)
    return y, mag


def packed_attention(q, k_cache, v_cache, cu_q, tables, lens, scale):
    """Row by row of each sequence, masked keys left out of every sum. Returns (out, sum p|v|) in float64."""
    T, Hq, d = q.shape
    NB, Hkv, bs, _ = k_cache.shape
    G = Hq // Hkv
    out = torch.zeros(T, Hq, d, dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(out)
    for b in range(len(cu_q) - 1):
        lo, hi, L = int(cu_q[b]), int(cu_q[b + 1]), int(lens[b])
        if hi == lo:
            continue
        ids = tables[b, :(L + bs - 1) // bs].long()
        K = k_cache[ids].permute(0, 2, 1, 3).reshape(-1, Hkv, d)[:L].double().repeat_interleave(G, 1)
        V = v_cache[ids].permute(0, 2, 1, 3).reshape(-1, Hkv, d)[:L].double().repeat_interleave(G, 1)
        for r in range(lo, hi, 256):
            e = min(hi, r + 256)
            s = torch.einsum("nhd,thd->hnt", q[r:e].double(), K) * scale
            pos = L - (hi - lo) + torch.arange(r - lo, e - lo, device=q.device)
            seen = torch.arange(L, device=q.device)[None, :] <= pos[:, None]
            p = torch.softmax(torch.where(seen, s, -math.inf), -1)
            # a value counts where its key is seen: nothing of the others reaches the row
            finite = torch.isfinite(V)
            out[r:e] = torch.einsum("hnt,thd->nhd", p, torch.where(finite, V, 0.0))
            mag[r:e] = torch.einsum("hnt,thd->nhd", p, torch.where(finite, V.abs(), 0.0))
            if not bool(finite.all()):
                for t, h, c in (~finite).nonzero().tolist():
                    out[r:e][pos >= t, h, c] += V[t, h, c]
    return out, mag


def adjusted(logits, history=None, history_lens=None, prompt_lens=None, draft=None, repetition=None, presence=None,
             frequency=None, bias_tokens=None, bias_values=None, mask=None):
    """Adjusted logits in float64 and the magnitude of the terms that each is made of."""
    B, R, V = logits.shape
    dev = logits.device
    out = torch.empty(B, R, V, dtype=torch.float64, device=dev)
    mag = torch.empty_like(out)
    for b in range(B):
        n = 0 if history is None else min(max(int(history_lens[b]), 0), history.shape[1])
        m = 0 if prompt_lens is None else int(prompt_lens[b])
        past = [] if history is None else history[b, :n].tolist()
        for j in range(R):
            made = past[max(m, 0):] + ([] if draft is None else draft[b, :j].tolist())
            count = torch.zeros(V, dtype=torch.float64)
            seen = torch.zeros(V, dtype=torch.bool)
            for t in made:
                if 0 <= t < V:
                    count[t] += 1
            for t in past:
                if 0 <= t < V:
                    seen[t] = True
            count, seen = count.to(dev), seen.to(dev)
            seen = seen | (count > 0)
            x = logits[b, j].double()
            w = x.abs()
            if repetition is not None:
                r = float(repetition[b])
                x = torch.where(seen, torch.where(x > 0, x / r, x * r), x)
                w = torch.maximum(w, x.abs())
            if frequency is not None:
                x = torch.where(count > 0, x - float(frequency[b]) * count, x)
                w = w + abs(float(frequency[b])) * count
            if presence is not None:
                x = torch.where(count > 0, x - float(presence[b]), x)
                w = w + abs(float(presence[b]))
            if bias_tokens is not None:
                bias = {}
                for t, v in zip(bias_tokens[b].tolist(), bias_values[b].tolist()):
                    if 0 <= t < V:
                        bias[t] = v
                for t, v in bias.items():
                    x[t] += v
                    w[t] += abs(v)
            if mask is not None:
                i = torch.arange(V, device=dev)
                ok = ((mask[b, j].long()[i // 32] >> (i % 32)) & 1) > 0
                x, w = torch.where(ok, x, -math.inf), torch.where(ok, w, 0.0)      # no term of a masked one counts
            out[b, j], mag[b, j] = x, w
    return out, mag


def probs(x, temperature):
    """The distribution of adjusted logits x [B, R, V] (float64)."""
    out = torch.zeros_like(x)
    for b in range(x.shape[0]):
        t = float(temperature[b])
        for j in range(x.shape[1]):
            row = x[b, j]
            if bool(torch.isnan(row).any()):
                out[b, j] = math.nan
            elif t == 0:
                m = row.max()
                if m > -math.inf:
                    out[b, j, int((row == m).nonzero()[0, 0])] = 1.0
            elif not t > 0:
                out[b, j] = math.nan
            elif float(row.max()) > -math.inf:
                e = torch.exp((row - row.max()) / t)
                out[b, j] = e / e.sum()
    return out
