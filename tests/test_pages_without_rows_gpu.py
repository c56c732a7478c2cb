"""Page tables of large admissions for callers that want no row lists, or short ones: the
entries against the sequential oracle, and their time beside that of the call with lists."""
import numpy as np
import pytest

import gpu_harness as H
from oracle import kv8

pytestmark = pytest.mark.gpu


class Step:
    def __init__(self, lens, new, max_pages, free, cursor, rows):
        t = H.torch()
        dev = lambda a: t.from_numpy(np.ascontiguousarray(a, np.int32)).to(H.DEV)  # noqa: E731
        b = len(lens)
        self.table = t.full((b, max_pages), -1, dtype=t.int32, device=H.DEV)
        self.lens, self.new, self.free, self.cursor = dev(lens), dev(new), dev(free), dev([cursor])
        self.after, self.page_starts, self.row_starts = (dev(np.full(n, 77)) for n in (b, b + 1, b + 1))
        self.seq_ids, self.positions, self.status = dev(np.full(rows, 77)), dev(np.full(rows, 77)), dev([0])

    def __call__(self, hold):
        H.lib().oscar_extend_pages(self.table, self.lens, self.new, self.free, self.cursor, self.after,
                                   self.page_starts, self.row_starts, self.seq_ids, self.positions,
                                   hold_back=hold, status=self.status)

    def check(self, want):
        H.torch().cuda.synchronize()
        got = (self.table, self.after, self.page_starts, self.row_starts, self.seq_ids, self.positions)
        for i, (x, y) in enumerate(zip(got, want)):
            np.testing.assert_array_equal(x.cpu().numpy(), y, err_msg=f"output {i}")


@pytest.mark.parametrize("rows", [0, 100])
@pytest.mark.parametrize("batch,lo,hi,hold,short", [
    (1, 140000, 140000, 0, 0),        # one sequence over many runs
    (256, 600, 640, 15, 0),           # a sequence ends inside every lane's run
    (4000, 0, 60, 0, 0),              # several sequences within 32 entries, and empty ones
    (40, 0, 9000, 128, 0),
    (40, 0, 9000, 15, 700),           # the free list ends 700 entries early
    (9, 131, 131072, 1, 12345),
])
def test_many_entries_match_the_sequential_list(batch, lo, hi, hold, short, rows):
    rng = np.random.default_rng(batch + hi)
    new = rng.integers(lo, hi + 1, batch)
    lens = np.zeros(batch, np.int64)
    need = sum(kv8.pages_held(n, hold) for n in new)
    assert need > 8192
    max_pages = -(-hi // 16)
    free = rng.permutation(need + 30)[:need + 5 - short]
    s = Step(lens, new, max_pages, free, 5, rows)
    s(hold)
    want = kv8.extend(np.full((batch, max_pages), -1), lens, new, free, 5, hold, rows)
    s.check(want)
    L = H.lib()
    assert H.status(s) == L.DEVERR_SEQ_LEN | (L.DEVERR_NO_PAGES if short else 0)


def test_many_entries_behind_what_the_sequences_hold():
    """Growth from ragged lengths, entries that were there kept, and a cursor carried on."""
    rng = np.random.default_rng(3)
    batch, hold, max_pages = 60, 15, 600
    lens, new = rng.integers(0, 900, batch), rng.integers(3000, 6000, batch)
    table, free, cursor = np.full((batch, max_pages), -1), rng.permutation(40000), 0
    for b in range(batch):
        for i in range(kv8.pages_held(lens[b], hold)):
            table[b, i], cursor = free[cursor], cursor + 1
    s = Step(lens, new, max_pages, free, cursor, 0)
    s.table.copy_(H.torch().from_numpy(table.astype(np.int32)))
    s(hold)
    s.check(kv8.extend(table, lens, new, free, cursor, hold, 0))


def test_tables_alone_take_no_multiple_of_tables_with_lists():
    """256 prompts of 4096 tokens.  Without lists one CTA writes the entries; with them a grid
    writes the entries and a million rows.  Measured 2.5 times; an entry at a time was 8 times."""
    t = H.torch()

    def best(rows):
        s = Step([0] * 256, [4096] * 256, 256, np.arange(256 * 256), 0, rows)
        s(15)
        graph = t.cuda.CUDAGraph()
        t.cuda.synchronize()
        with t.cuda.graph(graph):
            for _ in range(20):
                s(15)
        out = []
        for _ in range(8):
            a, b = t.cuda.Event(True), t.cuda.Event(True)
            a.record()
            graph.replay()
            b.record()
            t.cuda.synchronize()
            out.append(a.elapsed_time(b))
        return min(out)

    assert best(0) < 5 * best(256 * 4096)
