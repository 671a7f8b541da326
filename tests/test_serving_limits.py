"""More host-side refusals of the serving operators, and their limits as the header states them."""

import ctypes as C
import os
import re

import pytest

from paged_kv_cache_223_gb300 import _build


@pytest.fixture(scope="module")
def pa():
    _build.build_cuda()
    from paged_kv_cache_223_gb300 import pagedattn
    return pagedattn


@pytest.mark.parametrize("rot", [1, 17, 33, 127])
def test_a_base_gives_frequencies_of_whole_pairs(pa, rot):
    with pytest.raises(ValueError):
        pa.Rope.from_base(rot)


def header():
    text = open(os.path.join(_build.INCLUDE, "pagedattn.h")).read()
    return {n: int(v) for n, v in re.findall(r"#define (PA_\w+) (\d+)\n", text)}


@pytest.mark.parametrize("name,field", [("PA_LOGITS_MAX_VOCAB", "vocab"), ("PA_LOGITS_MAX_HISTORY", "history_stride"),
                                        ("PA_LOGITS_MAX_BIAS", "num_bias"), ("PA_LOGITS_MAX_ROWS", "rows_per_seq")])
def test_the_headers_limits_of_logits(pa, name, field):
    """The limit itself passes the checks (of a call without sequences), one more does not."""
    most = header()[name]
    for call in (pa._serving_lib().pa_adjust_logits, pa._serving_lib().pa_token_probs):
        for value, status in ((most, pa.PA_OK), (most + 1, pa.PA_ERR_UNSUPPORTED)):
            a = pa.PaLogitsArgs(dtype=2, num_seqs=0, rows_per_seq=1, vocab=100)
            setattr(a, field, value)
            assert call(C.byref(a), None) == status, (field, value)


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_the_headers_limit_of_frequencies(pa, sign):
    L, most, h = pa._serving_lib(), float(header()["PA_ROPE_MAX_FREQ"]), C.c_void_p()
    f = (C.c_double * 8)(*[sign * most] * 8)
    assert L.pa_rope_create(f, 16, 0, 1.0, 0, C.byref(h)) != pa.PA_ERR_INVALID_ARG       # without a GPU: PA_ERR_CUDA
    L.pa_rope_destroy(h)
    f[5] = sign * most * (1 + 2.0 ** -52)
    assert L.pa_rope_create(f, 16, 0, 1.0, 0, C.byref(h)) == pa.PA_ERR_INVALID_ARG and not h.value
