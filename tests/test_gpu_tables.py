"""pa_tables_grow and pa_tables_release against plain Python: page sizes, empty and long
requests, too few pages or rows, bad requests, slots listed twice, large calls, graphs."""
import random

import pytest
import torch

import paged_kv_continuous_pa_gb300 as pa
import serving_ref as R

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class State:
    def __init__(self, seqs, blocks, page, lengths, seed=0, spare=0):
        """Slots 0.. hold `lengths` tokens; the other pages are on the stack."""
        r = random.Random(seed)
        self.page, pages = page, sum(-(-n // page) for n in lengths) + spare
        order = list(range(pages))
        r.shuffle(order)
        self.tables = [[-1] * blocks for _ in range(seqs)]
        for s, n in enumerate(lengths):
            for c in range(-(-n // page)):
                self.tables[s][c] = order.pop()
        self.free, self.count, self.pages = order + [-1] * (pages - len(order)), len(order), pages


def grow(st, seq_ids, lengths, new, max_rows, count=None, in_place=False, slots=True):
    n = len(seq_ids)
    count = ints([st.count if count is None else count])
    left = count if in_place else ints([-5])
    t = dict(tables=ints(st.tables), row_starts=ints([-5] * (n + 1)), page_starts=ints([-5] * (n + 1)),
             seqs=ints([-5] * max_rows), pos=ints([-5] * max_rows),
             slots=torch.full((max_rows,), -5, dtype=torch.int64, device="cuda") if slots else None)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.tables_grow(ints(seq_ids), ints(lengths), ints(new), ints(st.free), count, left, st.page, t["tables"], t["row_starts"],
                   t["page_starts"], t["seqs"], t["pos"], row_slots=t["slots"], status=status)
    torch.cuda.synchronize()
    return t, int(left.item()), int(status.item())


def check(st, seq_ids, lengths, new, max_rows, **kw):
    t, left, status = grow(st, seq_ids, lengths, new, max_rows, **kw)
    tables, row_starts, page_starts, rows, want_left, want_status = R.grow(
        seq_ids, lengths, new, st.free, st.count, st.page, st.tables, max_rows)
    assert t["row_starts"].tolist() == row_starts and t["page_starts"].tolist() == page_starts
    assert t["tables"].tolist() == tables and left == want_left
    assert (status != 0) == (want_status != 0)
    rest = [-5] * (max_rows - len(rows))
    assert t["seqs"].tolist() == [r[0] for r in rows] + rest
    assert t["pos"].tolist() == [r[1] for r in rows] + rest
    if t["slots"] is not None:
        assert t["slots"].tolist() == [r[2] for r in rows] + rest
    return status


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_mixed_requests(page):
    lengths = [0, 1, page - 1, page, page + 1, 3 * page, 7, 0]
    new = [0, 1, 1, 1, 2 * page, 5, 0, 3 * page + 1]
    st = State(10, 9, page, lengths, seed=page, spare=20)
    order = [5, 2, 7, 0, 1, 4, 3, 6]
    for in_place in (False, True):
        assert check(st, order, [lengths[i] for i in order], [new[i] for i in order], 8 * page, in_place=in_place) == 0


@pytest.mark.parametrize("n", [1, 2, 31, 1023, 1024, 1025, 2500])
def test_decode_steps(n):
    r = random.Random(n)
    lengths = [r.randrange(0, 60) for _ in range(n)]
    st = State(n, 5, 16, lengths, seed=n, spare=n)
    assert check(st, list(range(n)), lengths, [1] * n, n, slots=n != 31) == 0


def test_prompts():
    """More rows than one CTA writes; the sums over several rounds."""
    r = random.Random(1)
    new = [r.randrange(0, 120) for _ in range(1500)]
    st = State(1500, 8, 16, [0] * 1500, spare=sum(-(-x // 16) for x in new))
    assert check(st, list(range(1500)), [0] * 1500, new, sum(new) + 3) == 0


def test_one_long_request():
    st = State(3, 4000, 16, [0, 0, 0], spare=4000)
    assert check(st, [1], [0], [63999], 64000) == 0


@pytest.mark.parametrize("max_rows", [40, 5000])
def test_too_few_pages_or_rows(max_rows):
    """The first request that does not fit and those behind it get nothing."""
    lengths = [5, 16, 0, 3, 0]
    st = State(5, 4, 16, lengths, spare=3)
    assert check(st, [0, 1, 2, 3, 4], lengths, [11, 1, 20, 13, 17], max_rows) == pa.PA_ERR_NO_PAGES
    st = State(5, 4, 16, lengths, spare=30)
    assert check(st, [0, 1, 2, 3, 4], lengths, [11, 1, 20, 13, 0], 31) == pa.PA_ERR_NO_PAGES


@pytest.mark.parametrize("max_rows", [200, 5000])
def test_bad_requests(max_rows):
    """They take nothing; the others do."""
    lengths = [5, 16, 0, 3, 0, 2]
    st = State(6, 4, 16, lengths, spare=30)
    ids = [0, 6, -1, 1, 2, 2, 3, 4, 5]
    assert check(st, ids, [5, 1, 1, 16, 0, 0, -3, 0, 2], [2, 1, 1, 4, 7, 7, 1, 65, -2], max_rows) == pa.PA_ERR_OUT_OF_RANGE


@pytest.mark.parametrize("max_rows", [64, 5000])
def test_bad_stack(max_rows):
    st = State(2, 4, 16, [0, 0], spare=4)
    t, left, status = grow(st, [0], [0], [20], max_rows, count=9)  # higher than the pool
    assert status == pa.PA_ERR_OUT_OF_RANGE and left == 9 and t["row_starts"].tolist() == [0, 0]
    st.free[3] = 77
    t, left, status = grow(st, [0, 1], [0, 0], [20, 16], max_rows)
    assert status == pa.PA_ERR_OUT_OF_RANGE and left == 1
    assert t["tables"].tolist()[0][:2] == [-1, st.free[2]] and t["tables"].tolist()[1][0] == st.free[1]
    assert t["slots"].tolist()[:16] == [-1] * 16 and t["slots"].tolist()[16] == st.free[2] * 16


def test_nothing():
    st = State(2, 4, 16, [0, 0], spare=4)
    t, left, status = grow(st, [], [], [], 0, slots=False)
    assert (left, status, t["row_starts"].tolist()) == (4, 0, [0])


@pytest.mark.parametrize("page", [16, 64])
def test_release(page):
    """Back in reverse, so that the same requests get the same pages again."""
    r = random.Random(page)
    n = 70
    new = [r.randrange(0, 6 * page) for _ in range(n)]
    st = State(n + 3, 7, page, [0] * n, seed=1, spare=sum(-(-x // page) for x in new) + 5)
    ids = list(range(n + 2, 2, -1))
    t, left, _ = grow(st, ids, [0] * n, new, sum(new))
    free, count = ints(st.free), ints([left])
    tables, status = t["tables"].clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.tables_release(ints(ids), ints(new), free, count, page, tables, status=status)
    assert int(status.item()) == 0 and int(count.item()) == st.count
    assert tables.tolist() == st.tables and free.tolist() == st.free
    # a part of each
    keep = [r.randrange(0, x + 20) for x in new]
    free, count, tables = ints(st.free), ints([left]), t["tables"].clone()
    pa.tables_release(ints(ids), ints(new), free, count, page, tables, keep_tokens=ints(keep), status=status)
    want, back = t["tables"].tolist(), []
    for s, x, k in zip(ids, new, keep):
        for c in range(-(-min(k, x) // page), -(-x // page)):
            back.append(want[s][c])
            want[s][c] = -1
    assert tables.tolist() == want and int(count.item()) == left + len(back) and int(status.item()) == 0
    assert free.tolist()[left:left + len(back)] == back[::-1] and free.tolist()[:left] == st.free[:left]


def test_bad_releases():
    st = State(5, 4, 16, [20, 33, 16, 5], spare=2)
    st.tables[1][1] = 99
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    free, count, tables = ints(st.free), ints([st.count]), ints(st.tables)
    pa.tables_release(ints([0, 1, 9, 2, 2, 3, 4]), ints([20, 33, 1, 16, 16, 65, 0]), free, count, 16, tables, status=status)
    want = [list(x) for x in st.tables]
    want[0][:2] = [-1, -1]
    assert int(status.item()) == pa.PA_ERR_OUT_OF_RANGE and tables.tolist() == want
    assert int(count.item()) == st.count + 2 and free.tolist()[st.count:st.count + 2] == st.tables[0][1::-1]
    # more than the pool has
    status.zero_()
    count, tables = ints([st.pages - 1]), ints(st.tables)
    pa.tables_release(ints([0]), ints([20]), free, count, 16, tables, status=status)
    assert int(status.item()) == pa.PA_ERR_OUT_OF_RANGE and int(count.item()) == st.pages - 1
    assert tables.tolist() == st.tables


def test_graph():
    """A captured loop of decode steps that keeps its own counts."""
    n, page = 5, 16
    st = State(n, 6, page, [14] * n, spare=4 * n)
    lengths, count, tables = ints([14] * n), ints([st.count]), ints(st.tables)
    ids, new, free = ints(list(range(n))), ints([1] * n), ints(st.free)
    starts, pages, seqs, pos = (ints([0] * k) for k in (n + 1, n + 1, n, n))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pa.tables_grow(ids, lengths, new, free, count, count, page, tables, starts, pages, seqs, pos)
        lengths.add_(1)
    for i in range(40):
        graph.replay()
        torch.cuda.synchronize()
        assert pos.tolist() == [14 + i] * n
    held = [x for row in tables.tolist() for x in row if x >= 0]
    assert len(held) == n * 4 and len(set(held)) == len(held) and int(count.item()) == st.count - 3 * n
