"""prefill_packed where a long context stands beside much other work: nothing is cut, or the items are not sorted."""
import pytest
import torch

import test_gpu_packed as packed_test

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16

CASES = [
    # new, old, hq, hkv, d, dtype, bs, spare rows
    ([3000, 1, 2], [0, 20000, 40000], 32, 8, 128, BF, 16, 0),                 # a prompt and a decode step in one call
    ([512] + [1] * 39 + [1], [0] + [1000] * 39 + [30000], 32, 8, 128, FP, 32, 0),
    ([9, 7, 14], [6000, 9001, 12345], 32, 8, 128, BF, 16, 4066),              # few live rows of a padded call
    ([9, 7], [300, 0], 8, 4, 64, FP, 16, 9000),
    ([2000, 2200, 5], [0, 100, 18000], 32, 1, 128, BF, 32, 0),                # 526 items, the long one last
    ([2000, 2200, 5], [0, 100, 3000], 64, 2, 64, FP, 16, 11),
    ([1] * 599 + [1], [500] * 599 + [17000], 8, 1, 64, BF, 16, 0),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{i}-t{sum(c[0])}-h{c[2]}.{c[3]}-d{c[4]}" for i, c in enumerate(CASES)])
def test_parity(case):
    new, old, hq, hkv, d, dt, bs, spare = case
    made = packed_test.make(90 + CASES.index(case), new, old, hq, hkv, d, dt, bs, spare_rows=spare, first=3 if spare else 0)
    out = torch.full_like(made[1], 7.0)
    packed_test.check(*made, out=out)
    lo, hi = int(made[2][0]), int(made[2][-1])
    assert bool((out[:lo] == 7.0).all()) and bool((out[hi:] == 7.0).all())
