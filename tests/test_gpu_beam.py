"""pa_beam_select and pa_beam_reorder against plain references, and a short
beam search over a paged cache against one over whole copies."""
import pytest
import torch

import cache_ref as R
import paged_kv_continuous_pa_gb300 as pa

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def select(logits, scores, n_out, finished=None, end_token=0):
    n, b, v = logits.shape
    size = pa.beam_workspace_bytes(n, b, v, n_out)
    ws = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda").fill_(0xA5)  # scratch: any contents
    out = (torch.full((n, n_out), 99, dtype=torch.int32, device="cuda"),
           torch.full((n, n_out), 99, dtype=torch.int32, device="cuda"), torch.full((n, n_out), 99.0, device="cuda"))
    for _ in range(2):  # the workspace serves call after call
        pa.beam_select(logits, scores, *out, finished=finished, end_token=end_token, workspace=ws)
    torch.cuda.synchronize()
    return [x.cpu() for x in out]


def reference(logits, scores, n_out, finished=None, end_token=0):
    """float64 scores of the best continuations, ties by (beam, token)."""
    n, b, v = logits.shape
    parents = torch.full((n, n_out), -1, dtype=torch.int32)
    tokens, best = parents.clone(), torch.full((n, n_out), float("-inf"), dtype=torch.float64)
    x, cum = logits.cpu().double(), scores.cpu().double()
    for i in range(n):
        total = cum[i].view(b, 1) + torch.log_softmax(x[i], dim=1)
        total[torch.isinf(torch.logsumexp(x[i], dim=1)) | torch.isnan(torch.logsumexp(x[i], dim=1))] = float("-inf")
        total = torch.where(torch.isfinite(total), total, float("-inf"))
        if finished is not None:
            for j in range(b):
                if int(finished[i, j]):
                    total[j] = float("-inf")
                    total[j, 0] = cum[i, j] if torch.isfinite(cum[i, j]) else float("-inf")
        order = torch.sort(total.view(-1), descending=True, stable=True).indices[:n_out]
        for k, at in enumerate(order.tolist()):
            s = float(total.view(-1)[at])
            if s == float("-inf"):
                break
            beam = at // v
            parents[i, k], best[i, k] = beam, s
            tokens[i, k] = end_token if finished is not None and int(finished[i, beam]) else at % v
    return parents, tokens, best


def check(logits, scores, n_out, finished=None, end_token=0):
    parents, tokens, got = select(logits, scores, n_out, finished, end_token)
    want_p, want_t, want_s = reference(logits, scores, n_out, finished, end_token)
    assert torch.equal(parents, want_p) and torch.equal(tokens, want_t)
    none = torch.isinf(want_s)
    assert torch.equal(none, torch.isinf(got))
    # log-sum-exp: FP32 exponentials (a few 2^-22) and FP32 sums of at most vocab / 256 + 16 additions
    # (2^-24 each); the score is rounded to FP32 once
    bound = (16 + logits.shape[2] / 256) * 2.0 ** -24 * 4 + 2.0 ** -24 * want_s.abs()
    assert ((got.double() - want_s).abs() <= bound)[~none].all()


def make(n, b, v, dtype=torch.float32, seed=0, std=2.0):
    g = torch.Generator().manual_seed(seed)
    logits = (torch.randn(n, b, v, generator=g) * std).to(dtype).cuda()
    scores = -torch.rand(n, b, generator=g).mul(9).cuda()
    return logits, scores


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("v", [1, 2, 7, 64, 1000, 4097, 50001, 131071])
def test_vocabularies(dtype, v):
    logits, scores = make(3, 4, v, dtype, seed=v)
    check(logits, scores, 8)


@pytest.mark.parametrize("b,n_out", [(1, 1), (1, 2), (1, 64), (2, 4), (5, 5), (5, 10), (16, 32), (32, 64), (31, 33)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_beams(b, n_out, dtype):
    logits, scores = make(4, b, 3001, dtype, seed=b)
    check(logits, scores, n_out)


@pytest.mark.parametrize("groups", [1, 3, 200])
def test_groups(groups):
    logits, scores = make(groups, 3, 777, seed=groups)
    check(logits, scores, 6)


@pytest.mark.parametrize("offset,pad", [(0, 1), (1, 0), (3, 5), (5, 3)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_at_any_address(offset, pad, dtype):
    """Padded rows, and a first element off every wider alignment; what lies between is poison."""
    n, b, v = 3, 4, 2047
    room = torch.full((n * b * (v + pad) + offset,), float("nan"), dtype=dtype, device="cuda")
    logits, scores = make(n, b, v, dtype, seed=pad)
    view = room[offset:].view(n, b, v + pad)[:, :, :v]
    view.copy_(logits)
    check(view, scores, 8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties(dtype):
    """Equal logits: the lowest beam, then the lowest token."""
    logits = torch.zeros(2, 3, 9000, dtype=dtype, device="cuda")
    scores = torch.zeros(2, 3, device="cuda")
    check(logits, scores, 10)
    logits[:, :, 8000:8100] = 2.0
    logits[:, 1, 5] = 2.0
    check(logits, scores, 64)
    signed = torch.where(torch.arange(9000, device="cuda") % 2 == 0, 0.0, -0.0).to(dtype)
    check(signed.expand(2, 3, 9000).contiguous(), scores, 7)


def test_identical_beams():
    logits, scores = make(2, 1, 5000, seed=1)
    check(logits.expand(2, 4, 5000).contiguous(), scores[:, :1].expand(2, 4).contiguous(), 12)


def test_first_step():
    """One live beam: the others' scores are -infinity and offer nothing."""
    logits, scores = make(3, 4, 600, seed=2)
    scores[:, 1:] = float("-inf")
    check(logits, scores, 8)


def test_finished_beams():
    logits, scores = make(4, 5, 800, seed=3)
    finished = ints([[0, 1, 0, 0, 1], [1, 1, 1, 1, 1], [0, 0, 0, 0, 0], [7, 0, 0, -1, 0]])
    logits[0, 1] = float("nan")  # a finished beam's logits are not looked at
    scores[3, 0] = float("-inf")
    check(logits, scores, 10, finished, end_token=17)


def test_forbidden_tokens_and_dead_rows():
    logits, scores = make(6, 3, 300, seed=4)
    logits[0, :, 5:] = float("-inf")     # five tokens left, 15 continuations
    logits[1, 0] = float("-inf")         # nothing allowed
    logits[2, 1, 77] = float("nan")
    logits[3, 2, 5] = float("inf")
    scores[4, 1] = float("nan")
    logits[5] = torch.finfo(torch.float32).min  # the lowest value everywhere: an even row
    check(logits, scores, 20)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masks_of_the_lowest_value(dtype):
    logits, scores = make(2, 3, 5000, dtype, seed=5)
    logits[:, :, 100:] = torch.finfo(dtype).min
    check(logits, scores, 12)


def test_sorted_rows():
    """Ascending and descending rows: every tile, or none but the first, holds the best."""
    up = torch.linspace(-8, 8, 40000, device="cuda").view(1, 1, -1)
    scores = torch.tensor([[0.0, -3.0]], device="cuda")
    check(torch.cat([up, up.flip(2)], dim=1).contiguous(), scores, 16)


def test_no_groups():
    e = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    pa.beam_select(torch.empty(0, 4, 10, device="cuda"), torch.empty(0, 4, device="cuda"), e, e.clone(),
                   torch.empty(0, 2, device="cuda"))


def test_select_in_a_graph():
    logits, scores = make(2, 4, 20000, torch.bfloat16, seed=6)
    size = pa.beam_workspace_bytes(2, 4, 20000, 8)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    parents, tokens = (torch.empty(2, 8, dtype=torch.int32, device="cuda") for _ in range(2))
    got = torch.empty(2, 8, device="cuda")
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pa.beam_select(logits, scores, parents, tokens, got, workspace=ws)
    for seed in (7, 8):
        fresh, s2 = make(2, 4, 20000, torch.bfloat16, seed=seed)
        logits.copy_(fresh)
        scores.copy_(s2)
        graph.replay()
        torch.cuda.synchronize()
        want = reference(fresh, s2, 8)
        assert torch.equal(parents.cpu(), want[0]) and torch.equal(tokens.cpu(), want[1])


# --------------------------------------------------------------- reorder --

def beam_cache(groups, beams, lengths, P=16, Hkv=2, D=64, kv="bf16", seed=0):
    """Slots of one group hold the same number of tokens; whole pages are shared at random."""
    per = [n for n in lengths for _ in range(beams)]
    c = R.make_cache([max(1, n) for n in per], Hkv=Hkv, D=D, P=P, kv=kv, seed=seed, spare_blocks=2)
    g = torch.Generator().manual_seed(seed + 1)
    for i, n in enumerate(lengths):
        rows = c.slots[i * beams:(i + 1) * beams]
        for j in range(n // P):
            own = c.tables[rows, j].clone()
            c.tables[rows, j] = own[torch.randint(0, beams, (beams,), generator=g).cuda()]
    return c


def reorder_and_check(c, groups, beams, lengths, parents, state=None):
    seq = torch.tensor(c.slots, dtype=torch.int32).view(groups, beams)
    tables, k, v = c.tables.clone(), c.k.clone(), c.v.clone()
    want_state = None if state is None else state.clone()
    for i, n in enumerate(lengths):
        whole, tail = divmod(n, c.P)
        for b in range(beams):
            me = int(seq[i, b])
            par = int(parents[i][b])
            src = int(seq[i, par]) if par >= 0 else me
            tables[me, :whole] = c.tables[src, :whole]
            if tail:
                to, at = int(c.tables[me, whole]), int(c.tables[src, whole])
                k[to, :, :tail], v[to, :, :tail] = c.k[at, :, :tail], c.v[at, :, :tail]
            if state is not None:
                want_state[me] = state[src]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.beam_reorder(c.pool, ints(parents), seq.cuda(), ints(lengths), c.tables, state=state, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(c.tables, tables)
    assert torch.equal(R.bits(c.k), R.bits(k)) and torch.equal(R.bits(c.v), R.bits(v))
    if state is not None:
        assert torch.equal(state, want_state)


@pytest.mark.parametrize("beams", [1, 2, 3, 4, 5, 8, 9, 16, 17, 32])
def test_reorder_beams(beams):
    g = torch.Generator().manual_seed(beams)
    lengths = [37, 64, 3, 0]
    c = beam_cache(4, beams, lengths, seed=beams)
    parents = torch.randint(0, beams, (4, beams), generator=g).tolist()
    reorder_and_check(c, 4, beams, lengths, parents)


@pytest.mark.parametrize("kind", ["swap", "rotate", "fan out", "own", "marked own", "last to all"])
def test_reorder_patterns(kind):
    beams = 6
    parents = {"swap": [1, 0, 3, 2, 5, 4], "rotate": [1, 2, 3, 4, 5, 0], "fan out": [0] * 6, "own": list(range(6)),
               "marked own": [-1, 0, -1, 2, -1, 1], "last to all": [5] * 6}[kind]
    c = beam_cache(2, beams, [100, 47], seed=3)
    state = torch.randn(c.num_seqs, 77, device="cuda")
    reorder_and_check(c, 2, beams, [100, 47], [parents, parents[::-1] if kind != "marked own" else parents], state)


@pytest.mark.parametrize("kv", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("D,P", [(64, 16), (128, 32), (128, 256)])
@pytest.mark.parametrize("fill", [0, 1, -1])
def test_reorder_pages(kv, D, P, fill):
    """A page boundary, one slot into a page, one short of a full page."""
    lengths = [2 * P + fill % P, fill % P]
    c = beam_cache(2, 4, lengths, P=P, D=D, kv=kv, seed=P)
    reorder_and_check(c, 2, 4, lengths, [[3, 3, 0, 1], [1, 2, 3, 0]])


@pytest.mark.parametrize("state_dtype,shape", [(torch.float32, (1,)), (torch.bfloat16, (2, 3, 5)), (torch.float32, (5000,)),
                                               (torch.uint8, (4,))])
def test_reorder_state(state_dtype, shape):
    c = beam_cache(2, 3, [20, 33], seed=4)
    state = torch.randn((c.num_seqs,) + shape, device="cuda").mul(50).to(state_dtype)
    if state.numel() // c.num_seqs * state.element_size() % 4:
        pytest.fail("the case's rows are a multiple of 4 bytes")
    reorder_and_check(c, 2, 3, [20, 33], [[2, 0, 0], [1, 1, 2]], state)


@pytest.mark.parametrize("what", ["slot", "parent", "length", "page", "slot twice", "page shared"])
def test_reorder_bad_groups(what):
    """A bad group is reported and left alone; the other one moves."""
    c = beam_cache(2, 3, [20, 33], seed=5)
    clean = beam_cache(2, 3, [20, 33], seed=5)
    seq = torch.tensor(c.slots, dtype=torch.int32).view(2, 3)
    parents, lengths = [[2, 0, 0], [1, 1, 2]], [20, 33]
    tables = c.tables
    if what == "slot":
        seq[0, 1] = c.num_seqs
    elif what == "parent":
        parents[0][2] = 3
    elif what == "length":
        lengths[0] = c.max_tokens + 1
    elif what == "page":
        tables[c.slots[1], 1] = c.k.shape[0]
    elif what == "slot twice":
        seq[0, 1] = seq[0, 0]
    else:
        tables[c.slots[1], 1] = tables[c.slots[0], 1]
    clean.tables.copy_(tables)
    reorder_and_check(clean, 2, 3, [20, 33], [[-1, -1, -1], parents[1]]) if what not in ("page", "page shared") else None
    k = c.k.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    before = tables.clone()
    pa.beam_reorder(c.pool, ints(parents), seq.cuda(), ints(lengths), tables, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == pa.PA_ERR_OUT_OF_RANGE
    assert torch.equal(tables[c.slots[:3]], before[c.slots[:3]])
    mine = c.tables[c.slots[:3]].long().clamp(0, c.k.shape[0] - 1)
    assert torch.equal(R.bits(c.k[mine]), R.bits(k[mine]))
    if what not in ("page", "page shared"):
        assert torch.equal(R.bits(c.k), R.bits(clean.k)) and torch.equal(tables, clean.tables)


# ------------------------------------------------------- a beam search --

def test_beam_search_over_a_paged_cache():
    """Steps of append + attention + selection + reordering, against the same
    search that keeps a whole K and V per hypothesis.  The `model` projects the
    attention output; its logits come from the library's attention in one search
    and from a 64-bit one in the other, so the test follows the paged search's
    choices and checks every step's inputs and moves."""
    beams, P, Hkv, G, D, V, steps, prompt = 4, 16, 2, 2, 64, 300, 40, 21
    g = torch.Generator().manual_seed(9)
    table_k, table_v = (torch.randn(V, Hkv, D, generator=g).bfloat16().cuda() for _ in range(2))
    table_q = torch.randn(V, Hkv * G, D, generator=g).bfloat16().cuda()
    head = torch.randn(Hkv * G * D, V, generator=g).cuda()
    max_blocks = -(-(prompt + steps) // P)
    # every beam owns a table row of pages; the prompt sits in beam 0's
    tables = torch.arange(beams * max_blocks, dtype=torch.int32, device="cuda").view(beams, max_blocks)
    k_pool = torch.full((beams * max_blocks, Hkv, P, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    v_pool = k_pool.clone()
    pool = pa.Pool(k_pool, v_pool)
    text = torch.randint(0, V, (prompt,), generator=g)
    pa.append_kv(pool, table_k[text], table_v[text], torch.zeros(prompt, dtype=torch.int32, device="cuda"),
                 torch.arange(prompt, dtype=torch.int32, device="cuda"), tables)
    slots = torch.arange(beams, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    # fan out: every beam takes beam 0's prompt
    pa.beam_reorder(pool, torch.zeros(1, beams, dtype=torch.int32, device="cuda"), slots.view(1, beams), ints([prompt]),
                    tables, status=status)
    hyps = [text.tolist() for _ in range(beams)]
    scores = torch.tensor([[0.0] + [float("-inf")] * (beams - 1)], device="cuda")
    last = torch.tensor([hyps[0][-1]] * beams)
    parents, tokens = (torch.empty(1, beams, dtype=torch.int32, device="cuda") for _ in range(2))
    ws = torch.zeros(pa.beam_workspace_bytes(1, beams, V, beams), dtype=torch.uint8, device="cuda")
    moved = 0
    for step in range(steps):
        length = prompt + step
        q = table_q[last]
        out = torch.empty_like(q)
        pa.attention(pool, q, slots, torch.full((beams,), length - 1, dtype=torch.int32, device="cuda"), tables, out)
        torch.cuda.synchronize()
        for b in range(beams):  # attention over the hypothesis's own tokens
            kk, vv = table_k[hyps[b]].double().transpose(0, 1), table_v[hyps[b]].double().transpose(0, 1)
            s = torch.einsum("hgd,htd->hgt", q[b].double().view(Hkv, G, D), kk) / D ** 0.5
            ref = torch.einsum("hgt,htd->hgd", torch.softmax(s, dim=2), vv).reshape(Hkv * G, D)
            err = (out[b].double() - ref).abs()
            assert ((err <= 2e-3) | (err <= 1e-2 * ref.abs())).all(), (step, b)
        logits = (out.float().view(beams, -1) @ head).view(1, beams, V)
        want = reference(logits, scores, beams)
        new_scores = torch.empty_like(scores)
        pa.beam_select(logits, scores, parents, tokens, new_scores, workspace=ws)
        assert torch.equal(parents.cpu(), want[0]) and torch.equal(tokens.cpu(), want[1])
        pa.beam_reorder(pool, parents, slots.view(1, beams), ints([length]), tables, status=status)
        choice, words = parents.cpu()[0].tolist(), tokens.cpu()[0].tolist()
        moved += sum(c != b for b, c in enumerate(choice))
        hyps = [hyps[p] + [w] for p, w in zip(choice, words)]
        last = torch.tensor(words)
        pa.append_kv(pool, table_k[last], table_v[last], slots, torch.full((beams,), length, dtype=torch.int32, device="cuda"),
                     tables, status=status)
        scores = new_scores
    assert int(status.item()) == 0 and moved > steps // 4


@pytest.mark.parametrize("b", [1, 4, 32])
def test_scores_in_place(b):
    """As many continuations as beams: the new scores may take the old ones' place."""
    logits, scores = make(5, b, 3001, seed=40 + b)
    want = reference(logits, scores, b)
    ws = torch.zeros(pa.beam_workspace_bytes(5, b, 3001, b), dtype=torch.uint8, device="cuda")
    parents, tokens = (torch.empty(5, b, dtype=torch.int32, device="cuda") for _ in range(2))
    apart = torch.empty_like(scores)
    pa.beam_select(logits, scores, parents, tokens, apart, workspace=ws)
    pa.beam_select(logits, scores, parents, tokens, scores, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(parents.cpu(), want[0]) and torch.equal(tokens.cpu(), want[1]) and torch.equal(scores, apart)


def test_calls_that_share_a_workspace():
    """Ruled out where they overlap, and their results unspecified: but nothing else is touched, and the next call is right."""
    n, b, out = 16, 6, 12
    sizes, streams = (40001, 300, 9001), [torch.cuda.Stream() for _ in range(3)]
    ws = torch.empty(max(pa.beam_workspace_bytes(n, b, v, out) for v in sizes), dtype=torch.uint8, device="cuda").fill_(0xA5)
    jobs, room = [], torch.full((3, 3, 3, n, out), -7, dtype=torch.int32, device="cuda")
    for i, v in enumerate(sizes):
        logits, scores = make(n, b, v, seed=50 + i, std=0.0 if i == 1 else 2.0)
        jobs.append((logits, scores, room[i, 1, 0], room[i, 1, 1], room[i, 1, 2].view(torch.float32)))
    torch.cuda.synchronize()
    for _ in range(60):
        for s, job in zip(streams, jobs):
            pa.beam_select(*job, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert (room[:, 0] == -7).all() and (room[:, 2] == -7).all()
    for logits, scores, parents, tokens, got in jobs:
        want = reference(logits, scores, out)
        pa.beam_select(logits, scores, parents, tokens, got, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(parents.cpu(), want[0]) and torch.equal(tokens.cpu(), want[1])
