"""The step's page tables against a sequence-by-sequence form on host lists (GPU)."""
from __future__ import annotations

import random

import pytest
import torch

import paged_attention_decode_kv_gb300 as vt
from drafts import pages, step

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module", autouse=True)
def dev():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    from paged_attention_decode_kv_gb300 import build_lib
    build_lib.build()
    vt.library()


def make_state(lens, room, spare, seed=0):
    """Sequences of `lens` tokens on pages of a shuffled pool with `spare` free ones."""
    rng = random.Random(seed)
    pool = sum(pages(L) for L in lens) + spare
    ids = list(range(pool))
    rng.shuffle(ids)
    tables = []
    for L in lens:
        tables.append([ids.pop() for _ in range(pages(L))])
        tables[-1] += [-5] * (room - len(tables[-1]))
    return dict(lens=list(lens), tables=tables, free=ids, room=room, pool=pool)


class Device:
    """The same state on the GPU."""

    def __init__(self, s):
        self.tables = torch.tensor(s["tables"], **I32).view(len(s["lens"]), s["room"])
        self.lens = torch.tensor(s["lens"], **I32)
        self.free = torch.tensor(s["free"] + [-9] * (s["pool"] - len(s["free"])), **I32)
        self.counters = torch.tensor([len(s["free"]), 77], **I32)

    def step(self, keep, new, T, **kw):
        pos, slots = torch.full((T,), -3, **I32), torch.full((T,), -4, **I32)
        out = vt.step_tables(self.lens, torch.tensor(new, **I32), self.tables, self.free, self.counters, T,
                             keep_lens=None if keep is None else torch.tensor(keep, **I32), positions=pos, slots=slots,
                             **kw)
        assert out[1] is pos and out[2] is slots
        return [x.tolist() for x in out]


def check(s, d, keep, new, T):
    keep_list = list(s["lens"]) if keep is None else keep
    starts, positions, slots, refused = step(s, keep_list, new, T)
    got = d.step(keep, new, T)
    assert got[0] == starts
    live = starts[-1]
    assert got[1] == positions + [-3] * (T - live)
    assert got[2] == slots + [-4] * (T - live)
    assert d.lens.tolist() == s["lens"]
    assert d.counters.tolist() == [len(s["free"]), refused]
    assert d.free[:len(s["free"])].tolist() == s["free"]
    assert d.tables.tolist() == s["tables"]
    return starts


@pytest.mark.parametrize("B", [1, 2, 31, 33, 200, 1024, 1025, 3000])
def test_random_steps(B):
    """Several steps in a row: prompts, single tokens, drafts cut back, sequences that end, stacks that run out."""
    rng = random.Random(B)
    room = 12
    s = make_state([rng.randint(0, 150) for _ in range(B)], room, spare=rng.randint(0, 3 * B), seed=B)
    d = Device(s)
    for i in range(6):
        keep = [max(0, L - rng.choice([0, 0, 1, 5, 40, L])) for L in s["lens"]]
        new = [rng.choice([0, 1, 1, 7, 33, rng.randint(0, 200)]) for _ in range(B)]
        T = rng.choice([sum(new) + 3, sum(new), max(1, sum(new) // 2)])
        check(s, d, keep if i % 3 else None, new, T)


def test_edges_of_pages():
    lens = [0, 0, 0, 0, 31, 32, 33, 63, 64, 65]
    new = [0, 1, 32, 33, 1, 1, 1, 2, 0, 32]
    s = make_state(lens, 5, 20)
    check(s, Device(s), None, new, 110)


def test_a_long_prompt_beside_single_tokens():
    s = make_state([100] * 40 + [0] + [7] * 23, 9000, 8300)
    check(s, Device(s), None, [1] * 40 + [262144] + [1] * 23, 262144 + 70)


def test_sequences_keep_their_pages():
    """As many pages taken as given back: the same ones, in every sequence.  (The first step takes one more in the
    third and fourth sequence; a second of the same lengths gives back what it takes.)"""
    s = make_state([40, 70, 64, 100], 8, 3)
    d = Device(s)
    check(s, d, [30, 60, 60, 31], [20, 12, 30, 70], 200)
    before = [list(t) for t in s["tables"]]
    check(s, d, [30, 60, 60, 31], [20, 12, 30, 70], 200)
    assert [t[:pages(L)] for t, L in zip(s["tables"], s["lens"])] == [t[:pages(L)] for t, L in
                                                                     zip(before, s["lens"])]


def test_growth_ends_with_the_first_that_does_not_fit():
    s = make_state([10] * 5, 20, 4)
    d = Device(s)
    # pages: 1 and 2 of 4 taken, then 5 do not fit, and the single token behind them waits too
    starts = check(s, d, None, [40, 70, 160, 1, 0], 1000)
    assert starts == [0, 40, 110, 110, 110, 110] and d.counters.tolist()[1] == 2
    # rows: the second one's do not fit
    assert check(s, d, None, [1, 5, 1, 0, 1], 5) == [0, 1, 1, 1, 1, 1]
    # a table's row that is too short holds nobody else up
    assert check(s, d, None, [20 * 32, 1, 1, 1, 1], 700) == [0, 0, 1, 2, 3, 4]


def test_no_rows_at_all():
    s = make_state([50, 64], 4, 2)
    d = Device(s)
    assert check(s, d, [0, 33], [0, 0], 4) == [0, 0, 0]  # one ends, one is cut back
    assert check(s, d, None, [3, 1], 0) == [0, 0, 0]     # no room for rows


def test_no_sequences():
    d = Device(dict(lens=[], tables=[], free=[3, 4], room=2, pool=5))
    assert d.step(None, [], 3) == [[0], [-3] * 3, [-4] * 3]
    assert d.counters.tolist() == [2, 0]


def test_as_many_sequences_as_are_taken():
    rng = random.Random(5)
    B = 16384
    s = make_state([rng.randint(0, 40) for _ in range(B)], 3, B)
    check(s, Device(s), [max(0, L - rng.randint(0, 9)) for L in s["lens"]], [rng.randint(0, 3) for _ in range(B)],
          2 * B)


def test_lengths_that_are_none():
    """Negative or too long contexts, keeps and growths leave their sequence as it is, without rows."""
    s = make_state([40, 40, 40, 40, 40, 40], 4, 8)
    s["lens"][1], s["lens"][2] = -7, 129
    d = Device(s)
    check(s, d, [40, -7, 129, 41, -1, 40], [1, 1, 1, 1, 1, -2], 10)
    assert d.counters.tolist()[1] == 5 and d.lens.tolist() == [41, -7, 129, 40, 40, 40]


def test_extreme_lengths():
    big = 2 ** 31 - 1
    s = make_state([32, 32, 32], 4, 8)
    check(s, Device(s), None, [big, 1, big], 10)
    s = make_state([32] * 5, 4, 8)
    check(s, Device(s), [32, 0, big, 32, 32], [96, 96, 96, 97, 1], 200)


@pytest.mark.parametrize("count", [-5, 9, 2 ** 31 - 1])
def test_a_stack_that_is_none(count):
    """A size below 0 is 0, one above the pool the pool's; nothing is read or written outside the stack."""
    guard = torch.full((3, 8), -9, **I32)
    free = guard[1]
    free.copy_(torch.arange(8, **I32))
    tables, lens = torch.tensor([[20, 21, -5, -5]], **I32), torch.tensor([64], **I32)
    counters = torch.tensor([count, 0], **I32)
    starts, pos, slots = vt.step_tables(lens, torch.tensor([64], **I32), tables, free, counters, 64,
                                        keep_lens=torch.tensor([0], **I32))
    on_stack = max(0, min(count, 8))
    if on_stack == 0:    # the sequence's own two pages come back to it
        assert tables.tolist() == [[20, 21, -5, -5]] and counters.tolist() == [0, 0]
    else:                # two more than the pool has are not kept
        assert tables.tolist() == [[7, 6, -5, -5]] and counters.tolist() == [6, 0]
    assert pos.tolist() == list(range(64)) and lens.tolist() == [64] and starts.tolist() == [0, 64]
    page = tables[0, 0].item()
    assert slots[0].item() == (page * 32 if page < 8 else -1)   # 20 and 21 are no pages of this pool
    assert (guard[0] == -9).all() and (guard[2] == -9).all()


def test_allocates_what_is_not_given_and_takes_a_stream():
    s = make_state([5, 60], 4, 5)
    d = Device(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    new = torch.tensor([2, 9], **I32)
    starts, pos, slots = vt.step_tables(d.lens, new, d.tables, d.free, d.counters, 11, stream=side)
    side.synchronize()
    want = step(s, list(s["lens"]), [2, 9], 11)
    assert [starts.tolist(), pos.tolist(), slots.tolist()] == list(want[:3])


def test_optional_outputs():
    s = make_state([5, 60], 4, 5)
    d = Device(s)
    new, starts = torch.tensor([30, 9], **I32), torch.zeros(3, **I32)
    st = vt.vt_paged_step_tables(d.tables.data_ptr(), d.lens.data_ptr(), d.free.data_ptr(), d.counters.data_ptr(),
                                 starts.data_ptr(), None, None, None, new.data_ptr(), 2, 39, 32,
                                 torch.cuda.current_stream().cuda_stream, 4, s["pool"])
    assert st == vt.VT_OK
    want = step(s, list(s["lens"]), [30, 9], 39)
    assert starts.tolist() == want[0] and d.tables.tolist() == s["tables"] and d.lens.tolist() == s["lens"]


def test_captured_and_replayed():
    """A graph of the step runs on from state to state."""
    s = make_state([5, 60, 0], 40, 60)
    d = Device(s)
    new, keep = torch.tensor([3, 17, 40], **I32), torch.zeros(3, **I32)
    starts, pos, slots = torch.zeros(4, **I32), torch.zeros(64, **I32), torch.zeros(64, **I32)
    kw = dict(q_starts=starts, positions=pos, slots=slots)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        vt.step_tables(d.lens, new, d.tables, d.free, d.counters, 64, **kw)
    for i in range(4):
        graph.replay()
        want = step(s, list(s["lens"]), [3, 17, 40], 64)
        n = want[0][-1]
        assert starts.tolist() == want[0] and pos.tolist()[:n] == want[1] and slots.tolist()[:n] == want[2]
        assert d.tables.tolist() == s["tables"]


def test_refusals():
    i = torch.zeros(4, **I32)
    table = torch.zeros((4, 2), **I32)
    free = torch.zeros(9, **I32)
    two = torch.zeros(2, **I32)
    with pytest.raises(TypeError):
        vt.step_tables(i.long(), i, table, free, two, 4)
    with pytest.raises(ValueError):
        vt.step_tables(i, i[:3], table, free, two, 4)
    with pytest.raises(ValueError):
        vt.step_tables(i, i, table, free, i, 4)
    with pytest.raises(ValueError):
        vt.step_tables(i, i, table[:3], free, two, 4)
    with pytest.raises(ValueError):
        vt.step_tables(i, i, table, free, two, 4, keep_lens=two)
    with pytest.raises(ValueError):
        vt.step_tables(i, i, table, free, two, 4, positions=i[:3])
    with pytest.raises(ValueError):
        vt.step_tables(i, i, table, free[::2], two, 4)
    with pytest.raises(vt.VtError):
        vt.step_tables(i, i, table, free[:0], two, 4)
    with pytest.raises(vt.VtError):
        vt.step_tables(torch.zeros(16385, **I32), torch.zeros(16385, **I32), torch.zeros((16385, 1), **I32), free, two, 4)
