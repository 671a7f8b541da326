"""adjust_logits and token_probs against their definitions in 64 bits.

Tolerances, with u = 2^-24: an adjusted logit is at most four fp32 steps on terms of magnitude w (the sum
of the magnitudes involved), each within u w: 4 u w. A probability's exponent (x - max) / T carries the
errors of x and of the maximum and two roundings of its own, 12 u max(w) / T in all; the exponential and
the quotient are within 4 u, the sum of non-negative terms in blocks within 64 u.
"""
import math

import pytest
import torch

from paged_kv_cache_223_gb300 import pagedattn as pa
from serving_reference import adjusted, probs

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
U = 2.0 ** -24


def make(seed, B, R, V, dt=torch.float32, S=50, NB=5, mask=True, draft=True, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *s: torch.rand(s, generator=g, device=DEV)  # noqa: E731
    full = (torch.randn(B, R, V + pad, generator=g, device=DEV) * 3).to(dt)
    ids = lambda *s: (rand(*s) ** 3 * (V + 2)).to(torch.int32) - 1  # noqa: E731  some are outside the vocabulary
    kw = {}
    if S:
        kw.update(history=ids(B, S), history_lens=torch.randint(-1, S + 2, (B,), generator=g, device=DEV,
                                                                dtype=torch.int32))
        kw["prompt_lens"] = torch.randint(-1, S + 2, (B,), generator=g, device=DEV, dtype=torch.int32)
    if draft and R > 1:
        kw["draft"] = ids(B, R - 1)
    kw.update(repetition=0.8 + rand(B), presence=rand(B) - 0.3, frequency=rand(B) - 0.3)
    if NB:
        kw.update(bias_tokens=ids(B, NB), bias_values=torch.randn(B, NB, generator=g, device=DEV) * 4)
    if mask:
        kw["mask"] = torch.randint(-2 ** 31, 2 ** 31, (B, R, (V + 31) // 32), generator=g, device=DEV,
                                   dtype=torch.int64).to(torch.int32)
    return full[:, :, :V], kw, 0.5 + rand(B)


def close_adjusted(out, ref, mag):
    assert torch.equal(torch.isneginf(out), torch.isneginf(ref))
    fine = torch.isfinite(ref)
    err = (out.double() - ref).abs()[fine]
    assert bool((err <= 4 * U * mag[fine] * 1.01).all()), float((err / (U * mag[fine] + 1e-30)).max())


def close_probs(out, ref, mag, t):
    for b in range(out.shape[0]):
        w = float(mag[b].max())
        rel = 12 * U * w / float(t[b]) + 80 * U if float(t[b]) > 0 else 0.0
        err = (out[b].double() - ref[b]).abs()
        assert bool((err <= rel * ref[b] + 2.0 ** -126).all()), (b, float((err / (ref[b] + 1e-300)).max()), rel)


CASES = [
    # B, R, V, dtype, S, NB, mask, draft, pad
    (1, 1, 1, torch.float32, 3, 1, False, False, 0),
    (1, 1, 31, torch.float32, 10, 3, True, False, 0),
    (2, 3, 33, torch.bfloat16, 40, 5, True, True, 1),
    (3, 1, 1000, torch.float16, 200, 0, False, False, 0),
    (1, 1, 32000, torch.float32, 300, 8, False, False, 0),
    (5, 6, 4099, torch.float32, 64, 20, True, True, 0),
    (2, 2, 50257, torch.float16, 500, 300, True, True, 7),
    (4, 2, 128256, torch.bfloat16, 1000, 30, True, True, 0),
    (2, 1, 128256, torch.float32, 0, 0, True, False, 64),
    (1, 2, 262144, torch.bfloat16, 100, 3, True, True, 0),
    (1, 1, 393216, torch.float32, 100, 3, False, False, 0),
    (170, 1, 700, torch.float32, 30, 3, True, False, 0),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}x{c[1]}x{c[2]}" for c in CASES])
def test_parity(case):
    B, R, V, dt, S, NB, mask, draft, pad = case
    logits, kw, t = make(7 + CASES.index(case), B, R, V, dt, S, NB, mask, draft, pad)
    ref, mag = adjusted(logits, **kw)
    close_adjusted(pa.adjust_logits(logits, **kw), ref, mag)
    close_probs(pa.token_probs(logits, t, **kw), probs(ref, t), mag, t)


@pytest.mark.parametrize("V", [9100, 9500, 36800, 40000, 72960, 76032, 79400])
def test_slices_whose_table_ends_near_48_kb(V):
    """Tables that reach the shared memory a launch has by default only together with the kernel's fixed part."""
    logits, kw, t = make(29, 2, 1, V, torch.float32, 100, 9, True, False, 0)
    ref, mag = adjusted(logits, **kw)
    close_adjusted(pa.adjust_logits(logits, **kw), ref, mag)
    close_probs(pa.token_probs(logits, t, **kw), probs(ref, t), mag, t)
    many = make(30, 320, 1, V, torch.bfloat16, 20, 2, False, False, 0)       # rows that fill the GPU: fewest slices
    ref, mag = adjusted(many[0], **many[1])
    close_adjusted(pa.adjust_logits(many[0], **many[1]), ref, mag)


@pytest.mark.parametrize("left_out", ["history", "repetition", "presence", "frequency", "bias", "mask", "draft",
                                      "prompt_lens", "all"])
def test_each_list_may_be_missing(left_out):
    logits, kw, t = make(30, 3, 3, 5000, S=200)
    gone = {"history": ["history", "history_lens", "prompt_lens"], "bias": ["bias_tokens", "bias_values"],
            "all": list(kw)}.get(left_out, [left_out])
    for k in gone:
        kw.pop(k)
    ref, mag = adjusted(logits, **kw)
    close_adjusted(pa.adjust_logits(logits, **kw), ref, mag)
    close_probs(pa.token_probs(logits, t, **kw), probs(ref, t), mag, t)


def test_greedy_rows_take_the_lowest_of_equals():
    logits, kw, t = make(31, 6, 2, 9000, torch.bfloat16, NB=0)
    t[::2] = 0.0
    logits[0, 0, :] = 1.0                              # all equal
    logits[2, 1, 4000] = logits[2, 1, 8999] = logits[2, 1, 4001] = 100.0
    for k in ("mask", "history", "history_lens", "prompt_lens", "draft"):
        kw.pop(k)
    out = pa.token_probs(logits, t, **kw)
    ref, mag = adjusted(logits, **kw)
    want = probs(ref, t)
    assert torch.equal(out[::2].double(), want[::2])
    assert float(out[0, 0, 0]) == 1.0 and float(out[2, 1, 4000]) == 1.0
    close_probs(out[1::2], want[1::2], mag[1::2], t[1::2])


def test_masks_that_leave_nothing_or_one():
    logits, kw, t = make(32, 4, 2, 3000)
    kw["mask"].zero_()
    kw["mask"][1, 1, 7] = 1 << 5
    t[2] = 0.0
    out = pa.token_probs(logits, t, **kw)
    assert float(out[1, 1, 7 * 32 + 5]) == 1.0 and float(out.sum()) == 1.0
    adj = pa.adjust_logits(logits, **kw)
    assert int(torch.isfinite(adj).sum()) == 1
    # rows without mass draw no token, one-token rows draw that token
    p = out[1:2].contiguous()
    tok, n = pa.spec_verify(p, p[:, :1].contiguous(), torch.tensor([[3]], dtype=torch.int32, device=DEV),
                            torch.tensor([[0.5]], device=DEV), torch.tensor([0.5], device=DEV))
    assert tok.tolist()[0][0] == -1


def test_values_that_are_no_numbers():
    logits, kw, t = make(33, 4, 1, 3000, NB=0)
    for k in ("history", "history_lens", "prompt_lens"):
        kw.pop(k)
    kw["mask"].fill_(-1)
    kw["mask"][:, :, 2] = 0
    logits[:, :, 64], logits[:, :, 65], logits[:, :, 66] = math.nan, math.inf, -math.inf
    ref, mag = adjusted(logits, **kw)
    close_probs(pa.token_probs(logits, t, **kw), probs(ref, t), mag, t)
    logits[0, 0, 5] = math.nan
    logits[1, 0, 5] = math.inf
    logits[2, 0, 5] = math.nan
    logits[3, 0, 5] = math.inf
    t[2] = t[3] = 0.0
    out = pa.token_probs(logits, t, **kw)
    assert bool(torch.isnan(out[:3]).all())
    assert float(out[3, 0, 5]) == 1.0 and float(out[3].sum()) == 1.0
    logits[:, :, 5] = torch.finfo(torch.float32).min          # the type's lowest value is a logit like others
    t.copy_(torch.tensor([1e-40, 3e38, -1.0, math.nan]))
    out = pa.token_probs(logits, t, **kw)
    live = torch.ones(3000, dtype=torch.bool, device=DEV)
    live[64:96] = False
    assert float(out[0].sum()) == 1.0 and bool(torch.isnan(out[2:]).all())
    assert abs(float(out[1, 0, 100]) - 1.0 / int(live.sum())) < 1e-6 and float(out[1, 0, 64]) == 0.0


def test_the_same_token_many_times():
    logits, kw, t = make(34, 2, 3, 2000, S=4000, NB=50)
    kw["history"].fill_(17)
    kw["history_lens"].fill_(4000)
    kw["prompt_lens"].fill_(100)
    kw["draft"].fill_(17)
    kw["bias_tokens"].fill_(17)
    kw["bias_tokens"][:, -3:] = -1
    kw.pop("mask")
    ref, mag = adjusted(logits, **kw)
    close_adjusted(pa.adjust_logits(logits, **kw), ref, mag)


def test_in_place_strides_streams_and_graph():
    logits, kw, t = make(35, 3, 2, 4096)
    want, want_p = pa.adjust_logits(logits, **kw), pa.token_probs(logits, t, **kw)
    x = logits.clone()
    assert pa.adjust_logits(x, out=x, **kw) is x and torch.equal(x, want)
    x = logits.clone()
    pa.token_probs(x, t, out=x, **kw)
    assert torch.equal(x, want_p)
    odd = torch.empty(3 * 2 * 4111 + 5, device=DEV)[3:3 + 3 * 2 * 4111].view(3, 2, 4111)[:, :, :4096]
    odd.copy_(logits)
    # rows between vectors are summed in another order: held to the definition, not to the aligned rows' bits
    ref, mag = adjusted(logits, **kw)
    assert torch.equal(pa.adjust_logits(odd, **kw), want)
    close_probs(pa.token_probs(odd, t, **kw), probs(ref, t), mag, t)
    some = torch.empty(3, 9, 4096, device=DEV)                 # the last positions of a longer output
    some[:, 5:7] = logits
    assert torch.equal(pa.token_probs(some[:, 5:7], t, **kw), want_p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = pa.token_probs(logits, t, stream=s, **kw)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want_p)
    out = torch.empty_like(want_p)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.token_probs(logits, t, out=out, **kw)
    logits.mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, pa.token_probs(logits, t, **kw))


def test_refusals_on_the_host():
    logits, kw, t = make(36, 3, 2, 500)
    for change in (dict(history=kw["history"].long()), dict(history_lens=None), dict(history_lens=kw["history_lens"][:2]),
                   dict(draft=kw["history"]), dict(repetition=kw["repetition"].double()),
                   dict(mask=kw["mask"][:, :, :-1].contiguous()), dict(bias_values=None),
                   dict(bias_values=kw["bias_values"][:, 1:].contiguous()), dict(out=logits[:2]),
                   dict(out=torch.empty(3, 2, 500, dtype=torch.bfloat16, device=DEV)),
                   dict(presence=kw["presence"].cpu()), dict(history=None)):
        with pytest.raises(ValueError):
            pa.adjust_logits(logits, **{**kw, **change})
    with pytest.raises(ValueError):
        pa.token_probs(logits[:, :, ::2], t)
    with pytest.raises(ValueError):
        pa.token_probs(logits, None)
    with pytest.raises(ValueError):
        pa.token_probs(logits.double(), t)
    with pytest.raises(pa.PagedAttnError):                     # in place needs the output's layout
        x = torch.empty(3, 2, 600, device=DEV)[:, :, :500]
        a = torch.empty(3 * 2 * 600, device=DEV)
        x = a.view(3, 2, 600)[:, :, :500]
        pa.token_probs(x, t, out=a[:3000].view(3, 2, 500))
    with pytest.raises(pa.PagedAttnError):
        pa.token_probs(torch.empty(1, 1, 393217, device=DEV), t[:1])
    assert pa.token_probs(logits[:0], t[:0]).shape == (0, 2, 500)
