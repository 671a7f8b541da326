"""Host-side refusals of the serving operators: no GPU is touched before they return."""
import ctypes as C

import pytest

from paged_kv_cache_223_gb300 import _build


@pytest.fixture(scope="module")
def pa():
    _build.build_cuda()
    from paged_kv_cache_223_gb300 import pagedattn
    return pagedattn


def test_rope_create(pa):
    L = pa._serving_lib()
    h = C.c_void_p()
    f = (C.c_double * 64)(*[1.0] * 64)
    bad = [(None, 128, 0, 1.0, 0), (f, 0, 0, 1.0, 0), (f, 8, 0, 1.0, 0), (f, 40, 0, 1.0, 0), (f, 144, 0, 1.0, 0),
           (f, 128, 2, 1.0, 0), (f, 128, 0, float("nan"), 0), (f, 128, 0, float("inf"), 0), (f, 128, 0, 1.0, -1)]
    for args in bad:
        assert L.pa_rope_create(*args, C.byref(h)) == pa.PA_ERR_INVALID_ARG and not h.value
    assert L.pa_rope_create(f, 128, 0, 1.0, 0, None) == pa.PA_ERR_INVALID_ARG
    for w in (float("nan"), float("inf"), 1e7):
        f[3] = w
        assert L.pa_rope_create(f, 128, 0, 1.0, 0, C.byref(h)) == pa.PA_ERR_INVALID_ARG
    L.pa_rope_destroy(None)


def test_calls_without_a_pool(pa):
    L = pa._serving_lib()
    n = C.c_uint64()
    assert L.pa_rope_append(None, None, None, 0, None, 0, None, 0, None, None, 1, 1, None, 0, None, None,
                            None) == pa.PA_ERR_INVALID_ARG
    assert L.pa_prefill_packed_workspace(None, 1, 1, 8, 1, C.byref(n)) == pa.PA_ERR_INVALID_ARG
    assert L.pa_prefill_packed(None, None, None, None, None, None, 1, None, 1, 1, 8, 0.1, None, 0, None,
                               None) == pa.PA_ERR_INVALID_ARG


def logits_args(pa, **change):
    """Arguments that pass every check but for the change (addresses that nothing dereferences on the host)."""
    a = dict(logits=1024, dtype=2, num_seqs=2, rows_per_seq=2, num_bias=1, vocab=100, seq_stride=200, row_stride=100,
             history=1024, history_stride=4, history_lens=1024, prompt_lens=1024, draft=1024, repetition=1024,
             presence=1024, frequency=1024, bias_tokens=1024, bias_values=1024, mask=1024, temperature=1024, out=4096)
    a.update(change)
    return pa.PaLogitsArgs(*[a[n] for n, _ in pa.PaLogitsArgs._fields_])


def test_logits_arguments(pa):
    L = pa._serving_lib()
    for f in (L.pa_adjust_logits, L.pa_token_probs):
        assert f(None, None) == pa.PA_ERR_INVALID_ARG
        for change in (dict(num_seqs=-1), dict(rows_per_seq=0), dict(num_bias=-1), dict(vocab=0), dict(seq_stride=-1),
                       dict(row_stride=-8), dict(history_stride=-1), dict(dtype=3), dict(dtype=-1), dict(logits=None),
                       dict(out=None), dict(history_lens=None), dict(bias_tokens=None), dict(bias_values=None),
                       dict(logits=1026), dict(dtype=0, logits=1025), dict(mask=1027), dict(out=4098),
                       dict(out=1024, row_stride=104), dict(out=1024, seq_stride=208), dict(out=1024, dtype=1),
                       dict(out=1424), dict(out=1020), dict(out=1024 + 1596)):     # over some of the logits: 400 floats at 1024
            assert f(C.byref(logits_args(pa, **change)), None) == pa.PA_ERR_INVALID_ARG, change
        for change in (dict(vocab=393217), dict(history_stride=1000001), dict(num_bias=2001), dict(rows_per_seq=4097),
                       dict(num_seqs=1 << 23)):
            assert f(C.byref(logits_args(pa, **change)), None) == pa.PA_ERR_UNSUPPORTED, change
        assert f(C.byref(logits_args(pa, num_seqs=0, logits=None, out=None)), None) == pa.PA_OK
    assert L.pa_token_probs(C.byref(logits_args(pa, temperature=None)), None) == pa.PA_ERR_INVALID_ARG
