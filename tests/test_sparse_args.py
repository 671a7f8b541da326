"""Host-side refusals of the sparse decode step's calls without a GPU, and the binding against the header."""
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


def test_calls_without_a_pool(pa):
    L, n = pa._sparse_lib(), C.c_uint64()
    a = pa.PaTablesArgs(num_seqs=1, num_tokens=1, block_table_stride=1)
    assert L.pa_step_tables(None, C.byref(a), None) == pa.PA_ERR_INVALID_ARG
    assert L.pa_step_tables(None, None, None) == pa.PA_ERR_INVALID_ARG
    assert L.pa_key_bounds_size(None, C.byref(n)) == pa.PA_ERR_INVALID_ARG
    assert L.pa_key_bounds(None, None, None, None, 1, None, 1, 1, None, None) == pa.PA_ERR_INVALID_ARG
    assert L.pa_select_blocks(None, None, None, None, 1, None, 1, 8, 1, 8, 1, 2, None, None) == pa.PA_ERR_INVALID_ARG
    assert L.pa_decode_selected(None, None, None, None, None, 8, None, 1, None, 1, 8, 1, 0.1, None,
                                None) == pa.PA_ERR_INVALID_ARG


def test_the_arguments_are_the_headers(pa):
    """Names and order of pa_tables_args' fields."""
    text = open(os.path.join(_build.INCLUDE, "pagedattn.h")).read()
    body = re.search(r"typedef struct pa_tables_args \{(.*?)\} pa_tables_args;", text, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = re.findall(r"(\w+);", body)
    assert names == [n for n, _ in pa.PaTablesArgs._fields_]
    assert [C.sizeof(t) for _, t in pa.PaTablesArgs._fields_] == [4] * 3 + [8] * 9


def test_the_limits_are_the_headers(pa):
    """Beside the calls' own tests: the values that they use."""
    text = open(os.path.join(_build.INCLUDE, "pagedattn.h")).read()
    limits = {n: int(v) for n, v in re.findall(r"#define (PA_TABLES_\w+|PA_SELECT_\w+) (\d+)\n", text)}
    assert limits == dict(PA_TABLES_MAX_SEQS=8192, PA_TABLES_MAX_TOKENS=2 ** 29, PA_SELECT_MAX_BUDGET=4096,
                          PA_SELECT_MAX_BLOCKS=262144)
