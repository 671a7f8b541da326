"""step_tables (pa_step_tables) against the same step done on the host, one sequence after the other: whole numbers, equal."""
import ctypes as C
import random

import pytest
import torch

from paged_kv_cache_223_gb300 import pagedattn as pa
from sparse_reference import ceil_div, step_tables

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class State:
    """Sequences with blocks of their own, the rest on the stack in any order."""

    def __init__(self, lens, stride, num_blocks, bs, seed=0):
        rng = random.Random(seed)
        ids = list(range(num_blocks))
        rng.shuffle(ids)
        self.bs, self.stride, self.lens = bs, stride, list(lens)
        self.rows = []
        for n in lens:
            k = ceil_div(n, bs)
            self.rows.append(ids[:k] + [-7] * (stride - k))
            ids = ids[k:]
        self.num_free = len(ids)
        self.free = ids + [-9] * (num_blocks - len(ids))
        self.pool = pa.Pool(num_blocks, bs, 1, 64, max_seqs=1, max_context_len=512)
        self.t = dict(context_lens=i32(self.lens), block_tables=i32(self.rows).view(len(lens), stride),
                      free_blocks=i32(self.free), num_free=i32([self.num_free]))

    def call(self, new, num_tokens, keep=None, **kw):
        return self.pool.step_tables(i32(new), num_tokens=num_tokens, keep_lens=None if keep is None else i32(keep),
                                     **self.t, **kw)

    def expect(self, new, num_tokens, keep=None):
        """Moves the host's state on; what the call gives."""
        self.rows, self.lens, self.free, self.num_free, *out = step_tables(
            new, self.lens, self.rows, self.free, self.num_free, num_tokens, self.bs, keep)
        return out

    def check(self, got, want):
        assert self.t["block_tables"].tolist() == self.rows
        assert self.t["context_lens"].tolist() == self.lens
        assert self.t["num_free"].tolist() == [self.num_free]
        assert self.t["free_blocks"].tolist() == self.free
        for g, w in zip(got, want):
            assert g.tolist() == w


@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("b,new_hi,old_hi,cut", [(1, 1, 40, 0), (1, 0, 0, 0), (3, 70, 100, 40), (31, 1, 300, 5), (257, 6, 200, 8),
                                                 (512, 40, 0, 0), (513, 3, 33, 100), (1500, 100, 60, 60)])
def test_steps(bs, b, new_hi, old_hi, cut):
    """Three steps on end: prompts, rejected tokens and ended requests, single tokens."""
    rng = random.Random(b * bs + new_hi)
    stride = ceil_div(old_hi + 3 * new_hi, bs) + 1
    s = State([rng.randint(0, old_hi) for _ in range(b)], stride, b * stride + 5, bs, seed=b)
    for step in range(3):
        new = [rng.choice([0, rng.randint(0, new_hi), new_hi]) for _ in range(b)]
        keep = None
        if step:
            keep = [rng.choice([0, n, 10 ** 9, max(0, n - rng.randint(0, cut))]) for n in s.lens]
        total = sum(new) + rng.choice([0, 1, 77])
        got = s.call(new, total, keep)
        s.check(got, s.expect(new, total, keep))
        assert s.pool.check() == pa.PA_OK


def test_taking_back_and_again_gives_the_same_blocks():
    s = State([100, 0, 33, 64], 20, 90, 16)
    new = [50, 100, 1, 0]
    first = s.call(new, 151)
    tables = s.t["block_tables"].clone()
    free = s.t["free_blocks"].clone()
    for _ in range(3):
        again = s.call(new, 151, keep=[100, 0, 33, 64])
        assert torch.equal(s.t["block_tables"], tables) and torch.equal(s.t["free_blocks"], free)
        assert all(torch.equal(a, f) for a, f in zip(again, first))
    assert s.pool.check() == pa.PA_OK


def test_the_last_free_block_and_none():
    s = State([16, 15], 8, 4, 16)
    s.call([1, 18], 19)                                  # 17 and 33 tokens: one block and two more, two are free
    assert s.pool.check() == pa.PA_ERR_OOM
    s.check((), ())
    got = s.call([1, 17], 19)
    s.check(got, s.expect([1, 17], 19))
    assert s.num_free == 0 and s.pool.check() == pa.PA_OK
    before = {k: v.clone() for k, v in s.t.items()}
    cu, pos, slots = s.call([0, 16], 20)
    assert s.pool.check() == pa.PA_ERR_OOM and s.pool.check() == pa.PA_OK
    assert all(torch.equal(before[k], v) for k, v in s.t.items())
    assert cu.tolist() == [0, 0, 0] and pos.tolist() == [0] * 20 and slots.tolist() == [-1] * 20
    got = s.call([0, 16], 20, keep=[0, 32])              # room where the other one ends
    s.check(got, s.expect([0, 16], 20, keep=[0, 32]))
    assert s.pool.check() == pa.PA_OK


@pytest.mark.parametrize("what", ["new", "len", "keep", "long", "longer", "tokens", "free", "free_high", "returned"])
def test_lengths_that_do_not_fit_change_nothing(what):
    s = State([40, 17, 5], 4, 30, 16)
    new, keep, tokens = [1, 2, 3], [40, 17, 5], 10
    if what == "new":
        new[1] = -1
    elif what == "len":
        s.t["context_lens"][2] = -3
    elif what == "keep":
        keep[0] = -2 ** 31
    elif what == "long":
        new[0] = 25
    elif what == "longer":
        new = [2 ** 31 - 1] * 3
        tokens = 100
    elif what == "tokens":
        tokens = 5
    elif what == "free":
        s.t["num_free"][0] = -1
    elif what == "free_high":
        s.t["num_free"][0] = 31
    elif what == "returned":
        s.t["num_free"][0] = 30
        keep[0] = 0
    before = {k: v.clone() for k, v in s.t.items()}
    cu, pos, slots = s.call(new, tokens, keep)
    assert s.pool.check() == pa.PA_ERR_DEVICE_BOUNDS
    assert all(torch.equal(before[k], v) for k, v in s.t.items())
    assert cu.tolist() == [0] * 4 and pos.tolist() == [0] * tokens and slots.tolist() == [-1] * tokens
    assert s.pool.check() == pa.PA_OK


def test_an_id_outside_the_pool_is_flagged():
    s = State([20, 3], 6, 12, 16)
    s.t["block_tables"][0, 1] = 12
    s.t["free_blocks"][s.num_free - 1] = -5               # the next block that is taken
    cu, pos, slots = s.call([1, 20], 21)
    assert s.pool.check() == pa.PA_ERR_DEVICE_BOUNDS
    assert cu.tolist() == [0, 1, 21] and pos.tolist() == [20] + list(range(3, 23))
    assert slots.tolist()[0] == -1 and slots.tolist()[1:14] == [s.rows[1][0] * 16 + i for i in range(3, 16)]
    assert slots.tolist()[14:] == [-1] * 7


@pytest.mark.parametrize("spare", [0, 1, 2, 3, 40000])
def test_many_tokens(spare):
    """Above 32768 rows the tokens are written by a kernel of their own; refused steps and wrong ids there too."""
    new = [12345, 0, 1, 20431, 7]
    s = State([3, 100, 0, 17, 16], 1400, 2100, 16)
    s.t["block_tables"][1, 0] = 2100                      # not this step's
    s.rows[1][0] = 2100
    got = s.call(new, sum(new) + spare)
    s.check(got, s.expect(new, sum(new) + spare))
    assert s.pool.check() == pa.PA_OK
    before = {k: v.clone() for k, v in s.t.items()}
    for bad, status in (([-1, 0, 0, 0, 0], pa.PA_ERR_DEVICE_BOUNDS), ([0, 0, 0, 0, 2000 * 8], pa.PA_ERR_OOM)):
        cu, pos, slots = s.call(bad, 40001)
        assert s.pool.check() == status and cu.tolist() == [0] * 6
        assert not bool(pos.any()) and bool((slots == -1).all()) and all(torch.equal(before[k], v) for k, v in s.t.items())
    cu, pos, slots = s.call([0, 5, 0, 0, 0], 40000)       # behind 100 tokens: a block that is in order
    assert s.pool.check() == pa.PA_OK and slots[:5].tolist() == [s.rows[1][6] * 16 + i for i in range(4, 9)]
    s.t["block_tables"][1, 6] = -3
    cu, pos, slots = s.call([0, 5, 0, 0, 0], 40000, keep=[2 ** 30, 100, 2 ** 30, 2 ** 30, 2 ** 30])
    assert s.pool.check() == pa.PA_ERR_DEVICE_BOUNDS and slots[:5].tolist() == [-1] * 5 and pos[:5].tolist() == list(range(100, 105))


@pytest.mark.parametrize("off", [1, 2, 3])
def test_outputs_off_the_vectors(off):
    new = [700, 3, 9000]
    s = State([3, 100, 0], 700, 900, 16)
    buf = torch.full((9800,), -5, dtype=torch.int32, device=DEV)
    buf64 = torch.full((9800,), -5, dtype=torch.int64, device=DEV)
    n = sum(new) + 5
    got = s.call(new, n, positions=buf[off:off + n], slot_mapping=buf64[off:off + n])
    s.check(got, s.expect(new, n))
    for b in (buf, buf64):
        assert bool((b[:off] == -5).all()) and bool((b[off + n:] == -5).all())


def test_no_sequences_and_no_tokens():
    s = State([], 3, 4, 16)
    cu, pos, slots = s.call([], 5)
    assert cu.tolist() == [0] and pos.tolist() == [0] * 5 and slots.tolist() == [-1] * 5 and s.pool.check() == pa.PA_OK
    s = State([5, 0], 3, 4, 16)
    got = s.call([0, 0], 0)
    s.check(got, s.expect([0, 0], 0))
    assert s.pool.check() == pa.PA_OK


def test_the_most_sequences():
    n = 8192
    s = State([n % 7 for n in range(n)], 2, 3 * n, 16)
    new = [(5 * i) % 23 for i in range(n)]
    keep = [3] * n
    got = s.call(new, sum(new) + 3, keep)
    s.check(got, s.expect(new, sum(new) + 3, keep))
    assert s.pool.check() == pa.PA_OK
    with pytest.raises(pa.PagedAttnError):
        State([0] * (n + 1), 1, 4, 16).call([0] * (n + 1), 1)


def test_keep_and_new_may_be_the_lengths_themselves():
    s = State([5, 40], 8, 20, 16)
    got = s.pool.step_tables(s.t["context_lens"], num_tokens=45, keep_lens=s.t["context_lens"], **s.t)
    s.check(got, s.expect([5, 40], 45))
    assert s.pool.check() == pa.PA_OK


def test_refusals():
    s = State([5, 40], 8, 20, 16)
    L, t = pa._sparse_lib(), s.t
    new, cu, pos, slots = i32([1, 1]), i32([0] * 3), i32([0] * 8), torch.zeros(8, dtype=torch.int64, device=DEV)
    good = dict(num_seqs=2, num_tokens=8, block_table_stride=8, new_lens=new.data_ptr(), keep_lens=None,
                context_lens=t["context_lens"].data_ptr(), block_tables=t["block_tables"].data_ptr(),
                free_blocks=t["free_blocks"].data_ptr(), num_free=t["num_free"].data_ptr(), cu_q=cu.data_ptr(),
                positions=pos.data_ptr(), slot_mapping=slots.data_ptr())
    changes = [dict(num_seqs=-1), dict(num_tokens=-1), dict(block_table_stride=0)]
    changes += [{k: None} for k in good if k not in ("num_seqs", "num_tokens", "block_table_stride", "keep_lens")]
    changes += [{k: good[k] + 2} for k in ("new_lens", "context_lens", "positions", "slot_mapping", "cu_q")]
    changes += [dict(slot_mapping=good["slot_mapping"] + 4), dict(keep_lens=good["positions"]), dict(new_lens=good["num_free"]),
                dict(cu_q=good["block_tables"] + 60), dict(positions=good["slot_mapping"] + 60),
                dict(num_free=good["free_blocks"] + 76), dict(keep_lens=good["context_lens"] + 4)]
    for c in changes:
        a = pa.PaTablesArgs(**{**good, **c})
        assert L.pa_step_tables(s.pool.handle, C.byref(a), None) == pa.PA_ERR_INVALID_ARG, c
    for c in (dict(num_seqs=8193), dict(num_tokens=2 ** 29 + 1), dict(num_tokens=2 ** 31 - 1)):
        a = pa.PaTablesArgs(**{**good, **c})
        assert L.pa_step_tables(s.pool.handle, C.byref(a), None) == pa.PA_ERR_UNSUPPORTED
    call = lambda **kw: s.pool.step_tables(**{**dict(new_lens=new, num_tokens=8), **t, **kw})  # noqa: E731
    for kw in (dict(new_lens=new.long()), dict(new_lens=new.cpu()), dict(new_lens=new[:1]), dict(num_tokens=-1),
               dict(cu_q=cu[:2]), dict(positions=pos[:7]), dict(slot_mapping=pos), dict(free_blocks=t["free_blocks"][:5]),
               dict(keep_lens=i32([1])), dict(block_tables=t["block_tables"].t()), dict(num_free=i32([1, 2]))):
        with pytest.raises(ValueError):
            call(**kw)
    s.check((), ())


def test_captured_steps():
    """A decode loop of one token a sequence, replayed: the lengths and tables move on by themselves."""
    s = State([15, 31, 0], 8, 24, 16)
    new, keep = i32([1, 1, 1]), i32([2 ** 30] * 3)
    out = dict(cu_q=i32([0] * 4), positions=i32([0] * 4), slot_mapping=torch.zeros(4, dtype=torch.int64, device=DEV))
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        s.pool.step_tables(new, num_tokens=4, keep_lens=keep, **s.t, **out)
    for i in range(20):
        if i == 7:
            keep[1] = 3                                   # cut back between two replays
        elif i == 8:
            keep[1] = 2 ** 30
        g.replay()
        want = s.expect([1, 1, 1], 4, keep.tolist())
        s.check(out.values(), want)
    assert s.pool.check() == pa.PA_OK


def test_another_stream():
    s = State([5, 40], 8, 20, 16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = s.call([20, 3], 30, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    s.check(got, s.expect([20, 3], 30))
