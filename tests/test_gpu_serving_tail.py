"""A serving step whose arrays have more rows than its requests get: finished requests, requests
that find no pages.  What the rows behind the last one held must not reach the cache."""
import os
import re

import pytest
import torch

import paged_kv_continuous_pa_gb300 as pa
import serving_ref as R
import test_gpu_serving_run as S

pytestmark = pytest.mark.gpu
ints, zeros = S.ints, S.zeros
PAGE, BLOCKS, HQ, HKV, D = S.PAGE, S.BLOCKS, S.HQ, S.HKV, S.D


def test_readme_step_with_requests_that_find_no_pages():
    """README's example over arrays of zeros: slot 0 holds 40 tokens, the last two requests get nothing."""
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        block = next(b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "tables_release" in b)
    new, num_pages = [5, 20, 33, 100, 7], 100
    n_rows, n_seqs, served = sum(new), len(new), 58
    tables = torch.full((n_seqs, BLOCKS), -1, dtype=torch.int32, device="cuda")
    tables[0, :3] = ints([97, 98, 99])
    bf16 = dict(dtype=torch.bfloat16)
    a = dict(pa=pa, torch=torch, num_pages=num_pages, Hkv=HKV, Hq=HQ, D=D, P=PAGE, n_rows=n_rows, n_seqs=n_seqs,
             slots=torch.arange(n_seqs, dtype=torch.int32, device="cuda"), lengths=ints([40, 0, 0, 0, 0]), new_tokens=ints(new),
             free_pages=torch.arange(num_pages, dtype=torch.int32, device="cuda"), free_count=ints([9]),
             block_tables=tables, row_starts=zeros(n_seqs + 1), page_starts=zeros(n_seqs + 1), row_seqs=zeros(n_rows),
             row_positions=zeros(n_rows), qkv=S.projections(n_rows, 2), q_out=zeros(n_rows, HQ, D, **bf16),
             k_rows=zeros(n_rows, HKV, D, **bf16), v_rows=zeros(n_rows, HKV, D, **bf16), out=zeros(n_rows, HQ, D, **bf16))
    exec(block, a)
    at = [0, 5, 25, 58, 58, 58]
    assert a["row_starts"].tolist() == at and a["lengths"].tolist() == [45, 20, 33, 0, 0]
    # the cached tokens' ranges are as they were (zeros), those of the tokens behind them are not
    for x in a["ranges"]:
        assert (x[[97, 98]] == 0).all() and (x[99, :, :8] == 0).all() and (x[99, :, 13:] == 0).all()
        assert (x[99, :, 8:13, 0] > 0).all()
    assert (a["q_out"][served:] == 0).all() and (a["out"][served:] == 0).all()
    for x, y in zip(at, at[1:4]):
        want, size, _, big = R.causal(a["q_out"][x:y], a["k_rows"][x:y], a["v_rows"][x:y], R.scale_of(D))
        assert bool(((a["out"][x:y].double() - want).abs() <= R.causal_bound(want, size, D, y - x, big)).all())
    # every page comes back, those of the request that was served in part of the call among them
    assert (a["block_tables"] == -1).all() and a["free_count"].item() == 12
    assert sorted(a["free_pages"][:12].tolist()) == list(range(9)) + [97, 98, 99]


@pytest.mark.parametrize("kind", ["int4", "bf16"])
def test_captured_step_of_a_fixed_size(kind):
    """Fewer tokens than rows, none at all, several of one sequence, and in the end too few pages."""
    s, _ = S.start(kind)
    n, rows = len(S.PROMPTS), 2 * len(S.PROMPTS)
    s.count.fill_(4)  # the stack ends soon
    size = max(1, pa.workspace_bytes(s.pool, rows, HQ, BLOCKS))
    s.ws = zeros(size, dtype=torch.uint8)
    new, qkv = zeros(n), S.projections(rows, 1)
    starts, pages, seqs, positions = zeros(n + 1), zeros(n + 1), zeros(rows), zeros(rows)
    out, grown = zeros(rows, HQ, D, dtype=torch.bfloat16), zeros(1)

    def step():
        seqs.fill_(-1)
        pa.tables_grow(s.ids, s.lengths, new, s.free, s.count, s.count, PAGE, s.tables, starts, pages, seqs, positions,
                       status=grown)
        q = s.take_in(qkv, seqs, positions)
        pa.attention(s.pool, q, seqs, positions, s.tables, out, workspace=s.ws)
        s.lengths.add_(starts[1:] - starts[:-1])
        return q

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        q = step()
    refused = 0
    for t, more in enumerate([[1, 1, 1, 1, 1], [0, 0, 0, 0, 0], [2, 0, 3, 0, 1], [0, 1, 0, 0, 0], [2, 2, 2, 2, 2], [1, 2, 1, 2, 1]] +
                             [[2, 2, 2, 2, 2]] * 8):
        lengths, tables, count = s.lengths.tolist(), s.tables.tolist(), s.count.item()
        before = [s.cached(i, m) for i, m in enumerate(lengths)]
        want_tables, want_starts, _, want_rows, left, status = R.grow(list(range(n)), lengths, more, s.free.tolist(), count, PAGE,
                                                                     tables, rows)
        new.copy_(ints(more))
        qkv.copy_(S.projections(rows, 20 + t))
        grown.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = len(want_rows)
        assert s.tables.tolist() == want_tables and starts.tolist() == want_starts and s.count.item() == left
        assert grown.item() == status
        assert seqs.tolist() == [r[0] for r in want_rows] + [-1] * (rows - got)
        assert positions[:got].tolist() == [r[1] for r in want_rows]
        assert s.lengths.tolist() == [m + b - a for m, a, b in zip(lengths, want_starts, want_starts[1:])]
        for i, m in enumerate(lengths):
            assert all(x is y or torch.equal(x, y) for x, y in zip(s.cached(i, m)[:2], before[i][:2]))
        assert (out[got:] == 0).all()
        for r, (slot, position, _) in enumerate(want_rows):
            S.check_row(s, slot, position + 1, q[r], out[r])
        refused += status == pa.PA_ERR_NO_PAGES
    assert refused > 0
