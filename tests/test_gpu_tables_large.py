"""pa_tables_release of batches of many rounds of a CTA's warps, with requests of many columns, against plain Python; and
such a batch's pages taken again."""
import random

import pytest
import torch

import paged_kv_continuous_pa_gb300 as pa
import test_gpu_tables as T

pytestmark = pytest.mark.gpu
ints = T.ints


def release(ids, lengths, keep, free, count, page, tables, pages):
    """Plain Python on lists: (tables, free, count, refused)."""
    tables, back, refused = [list(x) for x in tables], [], False
    for s, x, k in zip(ids, lengths, keep):
        ok = 0 <= s < len(tables) and ids.count(s) == 1 and 0 <= x <= len(tables[0]) * page and k >= 0
        columns = range(-(-min(k, x) // page), -(-x // page)) if ok else ()
        if not ok or any(not 0 <= tables[s][c] < pages for c in columns):
            refused = True
            continue
        for c in columns:
            back.append(tables[s][c])
            tables[s][c] = -1
    free = list(free)
    free[count:count + len(back)] = back[::-1]
    return tables, free, count + len(back), refused


@pytest.mark.parametrize("n,longest", [(1023, 60), (1024, 100), (1025, 40), (2500, 90), (33, 3000)])
@pytest.mark.parametrize("partly", [False, True])
@pytest.mark.parametrize("bad", [0, 7])
def test_release(n, longest, partly, bad):
    r = random.Random(n + partly)
    page = 16
    lengths = [r.randrange(0, longest) * r.randrange(0, 2) for _ in range(n)]
    st = T.State(n + 5, -(-longest // page) + 1, page, lengths + [0] * 5, seed=n, spare=11)
    ids = list(range(n))
    r.shuffle(ids)
    size = [lengths[i] for i in ids]
    keep = [r.randrange(0, x + 20) if partly else 0 for x in size]
    for i in r.sample(range(n), bad):  # a page that is none, slots that are none or listed twice, a length that is too long
        kind = r.randrange(0, 4)
        if kind == 0 and size[i] > 0:
            st.tables[ids[i]][r.randrange(0, -(-size[i] // page))] = r.choice([-1, st.pages])
        elif kind == 1:
            ids[i] = r.choice([-1, n + 5])
        elif kind == 2:
            ids[i] = ids[(i + 1) % n]
        else:
            size[i] = len(st.tables[0]) * page + 1
    want_tables, want_free, want_count, refused = release(ids, size, keep, st.free, st.count, page, st.tables, st.pages)
    tables, free, count = ints(st.tables), ints(st.free), ints([st.count])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.tables_release(ints(ids), ints(size), free, count, page, tables, keep_tokens=ints(keep) if partly else None, status=status)
    assert tables.tolist() == want_tables and count.item() == want_count
    assert free.tolist()[:want_count] == want_free[:want_count]
    assert status.item() == (pa.PA_ERR_OUT_OF_RANGE if refused else 0)


def test_grown_again():
    """What a large batch gives back it gets again, page by page."""
    r = random.Random(1)
    n, page = 1500, 16
    new = [r.randrange(0, 200) for _ in range(n)]
    st = T.State(n, 13, page, [0] * n, seed=2, spare=sum(-(-x // page) for x in new) + 3)
    ids = list(range(n))
    r.shuffle(ids)
    t, left, status = T.grow(st, ids, [0] * n, new, sum(new))
    assert status == 0
    free, count, tables = ints(st.free), ints([left]), t["tables"].clone()
    pa.tables_release(ints(ids), ints(new), free, count, page, tables)
    assert count.item() == st.count and free.tolist() == st.free and (tables == -1).all()
    again, left2, status = T.grow(st, ids, [0] * n, new, sum(new))
    assert status == 0 and left2 == left and torch.equal(again["tables"], t["tables"])
