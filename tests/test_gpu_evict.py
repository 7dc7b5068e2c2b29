"""pa_evict_select and pa_evict_compact against plain references, and a run of
the whole: attend, accumulate weights, select, compact, trim, attend again."""
import numpy as np
import pytest
import torch

import cache_ref as R
import paged_kv_continuous_pa_gb300 as pa

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def select(mass, slots, lengths, budget, first=0, last=0):
    keep = torch.full((len(slots), mass.shape[1], budget), 77, dtype=torch.int32, device="cuda")
    kept = torch.full((len(slots),), 77, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.evict_select(mass, ints(slots), ints(lengths), keep, kept_lengths=kept, keep_first=first, keep_last=last,
                    status=status)
    torch.cuda.synchronize()
    return keep.cpu(), kept.cpu(), int(status.item())


def check_select(mass, slots, lengths, budget, first=0, last=0):
    keep, kept, status = select(mass.cuda(), slots, lengths, budget, first, last)
    assert status == 0
    assert kept.tolist() == [min(n, budget) for n in lengths]
    for i, (s, n) in enumerate(zip(slots, lengths)):
        for h in range(mass.shape[1]):
            want = R.select_ref(mass[s, h], n, budget, first, last)
            assert keep[i, h].tolist() == want + [-1] * (budget - len(want)), (i, h)


def weights(shape, kind, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "spread":
        return torch.randn(shape, generator=g).mul(4).exp()
    if kind == "ties":
        return torch.randint(0, 4, shape, generator=g).float()
    if kind == "equal":
        return torch.full(shape, 0.25)
    if kind == "signs":
        x = torch.randn(shape, generator=g)
        x[x.abs() < 0.3] = 0.0
        return torch.where(torch.rand(shape, generator=g) < 0.5, x, -x)  # -0 among them
    x = torch.randn(shape, generator=g)
    r = torch.rand(shape, generator=g)
    x[r < 0.2] = float("nan")
    x[(r >= 0.2) & (r < 0.3)] = float("-inf")
    x[(r >= 0.3) & (r < 0.4)] = float("inf")
    return x


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "signs", "special"])
@pytest.mark.parametrize("budget,first,last", [(1, 0, 0), (7, 2, 3), (64, 0, 16), (64, 64, 0), (64, 10, 54), (300, 4, 32)])
def test_select(kind, budget, first, last):
    mass = weights((5, 3, 700), kind, budget)
    check_select(mass, [4, 0, 2], [700, 65, 301], budget, first, last)


@pytest.mark.parametrize("length", [0, 1, 2, 63, 64, 65, 1023, 1024, 1025])
def test_select_lengths(length):
    mass = weights((2, 2, 1100), "spread", length)
    check_select(mass, [1], [length], 64, 2, 8)


@pytest.mark.parametrize("kind", ["spread", "ties", "equal"])
@pytest.mark.parametrize("length,budget", [(8193, 100), (20000, 4096), (40001, 39000), (140000, 1000)])
def test_select_long(kind, length, budget):
    mass = weights((2, 1, length), kind, length)
    check_select(mass, [1, 0], [length, length // 2 + 1], budget, 4, 64)


@pytest.mark.parametrize("kind", ["ascending", "descending", "steps", "last block", "stripes", "zeros"])
@pytest.mark.parametrize("budget", [10, 700, 8000])
def test_select_orders(kind, budget):
    """Orders that evenly spaced samples misjudge, and large groups of equal weights."""
    n = 20011
    t = torch.arange(n, dtype=torch.float32)
    w = {"ascending": t, "descending": -t, "steps": (t / 1000).floor(), "last block": (t >= n - 6000) * (t + 1),
         "stripes": (t % 40 < 2) * (t + 1), "zeros": (t % 7 == 0) * (t + 1)}[kind]
    check_select(torch.stack([w, w.flip(0)]).view(1, 2, n), [0], [n], budget, 3, 5)


@pytest.mark.parametrize("n", [90, 12000])
def test_select_between_kinds(n):
    """The last kept weight on every border: positive, zeros of both signs, negative, lowest, -infinity, NaN."""
    g = torch.Generator().manual_seed(n)
    parts = [torch.tensor([2.0, 1e-45, 0.0, -0.0, -1e-45, -3.0, torch.finfo(torch.float32).min, float("-inf"), float("nan")])]
    w = parts[0].repeat(n // 9 + 1)[:n][torch.randperm(n, generator=g)]
    mass = w.view(1, 1, n)
    for budget in sorted({1, n - 1} | {n * k // 9 + d for k in range(1, 9) for d in (-1, 0, 1)}):
        check_select(mass, [0], [n], budget)


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "signs", "special"])
@pytest.mark.parametrize("budget,first,last", [(1, 0, 0), (64, 10, 54), (3000, 4, 32), (20000, 0, 256)])
def test_select_wide_table(kind, budget, first, last):
    """Long tables: rows of every length in them, in few units and in many."""
    mass = weights((6, 2, 70003), kind, budget)
    check_select(mass, [4, 0, 2, 5, 1, 3], [70003, 33000, 0, 20001, 1, 20300], budget, first, last)


@pytest.mark.parametrize("kind", ["ascending", "stripes", "zeros"])
@pytest.mark.parametrize("budget", [700, 60000])
def test_select_wide_orders(kind, budget):
    n = 131101
    t = torch.arange(n, dtype=torch.float32)
    w = {"ascending": t, "stripes": (t % 40 < 2) * (t + 1), "zeros": (t % 7 == 0) * (t + 1)}[kind]
    check_select(torch.stack([w, w.flip(0)]).view(1, 2, n), [0], [n], budget, 3, 5)


def test_select_many_long_rows():
    mass = weights((160, 1, 33001), "spread", 3)
    lengths = [33001 - 7 * i for i in range(160)]
    check_select(mass, list(range(160)), lengths, 16000, 4, 64)


def test_select_many_rows():
    mass = weights((300, 2, 130), "ties", 1)
    lengths = [(i * 37) % 131 for i in range(300)]
    check_select(mass, list(range(299, -1, -1)), lengths, 40, 1, 5)


def test_select_bad_rows():
    mass = weights((3, 2, 50), "spread", 2)
    keep, kept, status = select(mass.cuda(), [0, 3, -1, 2, 1], [50, 10, 10, 51, -1], 8)
    assert status == pa.PA_ERR_OUT_OF_RANGE
    assert kept.tolist() == [8, 0, 0, 0, 0]
    assert (keep[1:] == -1).all() and (keep[0] >= 0).all()


# --------------------------------------------------------------- compact --

def random_keep(lengths, Hkv, budget, seed):
    g = torch.Generator().manual_seed(seed)
    keep = torch.full((len(lengths), Hkv, budget), -1, dtype=torch.int32)
    for i, n in enumerate(lengths):
        for h in range(Hkv):
            m = min(n, budget)
            keep[i, h, :m] = torch.randperm(n, generator=g)[:m].sort().values.to(torch.int32)
    return keep


def compact_and_check(c, keep, dst=None, with_mass=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    mass = torch.rand(c.num_seqs, c.Hkv, c.max_tokens, generator=g).cuda() if with_mass else None
    slots = c.slots[:keep.shape[0]]
    lengths = c.lengths[:keep.shape[0]]
    want_k, want_v, want_m = c.k.clone(), c.v.clone(), None if mass is None else mass.clone()
    into = slots if dst is None else dst
    for i, (s, to, n) in enumerate(zip(slots, into, lengths)):
        m = min(n, keep.shape[2])
        at = torch.arange(m, device="cuda")
        for h in range(c.Hkv):
            t = keep[i, h, :m].long().cuda()
            for new, old in ((want_k, c.k), (want_v, c.v)):
                new[c.tables[to][at // c.P].long(), h, at % c.P] = old[c.tables[s][t // c.P].long(), h, t % c.P]
            if mass is not None:
                want_m[to, h, m:n] = 0
                want_m[to, h, :m] = mass[s, h, t]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.evict_compact(c.pool, keep.cuda(), ints(slots), ints(lengths), c.tables, mass=mass,
                     dst_seq_ids=None if dst is None else ints(dst), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    assert torch.equal(R.bits(c.k), R.bits(want_k)) and torch.equal(R.bits(c.v), R.bits(want_v))
    if mass is not None:
        assert torch.equal(mass, want_m)


@pytest.mark.parametrize("kv", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [16, 256])
@pytest.mark.parametrize("copy", [False, True])
def test_compact(kv, D, P, copy):
    lengths = [700, 1, 100, 99, 513] + ([1] * 5 if copy else [])
    c = R.make_cache(lengths, Hkv=3, D=D, P=P, kv=kv, seed=P + D, slots=range(len(lengths)))
    compact_and_check(c, random_keep(lengths[:5], 3, 100, P), dst=list(range(9, 4, -1)) if copy else None)


@pytest.mark.parametrize("budget", [1, 2, 31, 64, 65, 1000, 4096])
def test_compact_budgets(budget):
    lengths = [5000, 1001, budget]
    c = R.make_cache(lengths, Hkv=2, D=128, P=32, seed=budget)
    compact_and_check(c, random_keep(lengths, 2, budget, budget))


def test_compact_one_long_sequence():
    c = R.make_cache([40000], Hkv=1, D=128, P=64, seed=1)
    compact_and_check(c, random_keep([40000], 1, 20000, 1), with_mass=False)


@pytest.mark.parametrize("kind", ["head", "tail", "one gap", "alternate"])
def test_compact_patterns(kind):
    """Shifts of one slot, no shift, the largest shift: where moving in place could tread on itself."""
    n, budget = 3001, 1500
    t = torch.arange(n)
    keep = {"head": t[:budget], "tail": t[-budget:], "one gap": torch.cat([t[:1], t[2:budget + 1]]),
            "alternate": t[::2][:budget]}[kind]
    c = R.make_cache([n, n], Hkv=2, D=64, P=32, seed=2)
    compact_and_check(c, keep.to(torch.int32).view(1, 1, -1).repeat(2, 2, 1))


def test_compact_empty_and_zero_length():
    c = R.make_cache([20, 20], Hkv=2, D=64, P=16, seed=3)
    before = c.k.clone()
    mass = torch.ones(c.num_seqs, 2, c.max_tokens, device="cuda")
    keep = torch.full((1, 2, 8), -1, dtype=torch.int32, device="cuda")
    pa.evict_compact(c.pool, keep, ints(c.slots[:1]), ints([0]), c.tables, mass=mass)
    pa.evict_compact(c.pool, keep[:0], ints([]), ints([]), c.tables, mass=mass)
    torch.cuda.synchronize()
    assert torch.equal(R.bits(before), R.bits(c.k)) and torch.equal(mass, torch.ones_like(mass))


@pytest.mark.parametrize("what", ["slot", "dst", "length", "order", "range", "page"])
def test_compact_bad_rows(what):
    """Whatever is wrong is reported, and other sequences' bytes stay or move as asked."""
    c = R.make_cache([100, 100], Hkv=2, D=64, P=16, seed=4)
    keep = random_keep([100, 100], 2, 20, 5)
    clean = R.make_cache([100, 100], Hkv=2, D=64, P=16, seed=4)
    compact_and_check(clean, keep, with_mass=False)
    slots, lengths, dst = list(c.slots), [100, 100], list(c.slots)
    tables = c.tables.clone()
    if what == "slot":
        slots[0] = c.num_seqs
    elif what == "dst":
        dst[0] = -2
    elif what == "length":
        lengths[0] = c.max_tokens + 1
    elif what == "order":
        keep[0, 1, 5] = keep[0, 1, 4]
    elif what == "range":
        keep[0, 0, 19] = 100
    else:
        tables[c.slots[0], 0] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.evict_compact(c.pool, keep.cuda(), ints(slots), ints(lengths), tables, dst_seq_ids=ints(dst), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == pa.PA_ERR_OUT_OF_RANGE
    other = c.tables[c.slots[1]].long()
    assert torch.equal(R.bits(c.k[other]), R.bits(clean.k[other]))
    rest = torch.ones(c.k.shape[0], dtype=torch.bool, device="cuda")
    rest[c.tables[c.slots[0]].long()] = False
    assert torch.equal(R.bits(c.k[rest]), R.bits(clean.k[rest]))


# ------------------------------------------------------------- the whole --

def attend(c, q, slots, lengths, tables):
    out = torch.empty_like(q)
    size = pa.workspace_bytes(c.pool, len(slots), q.shape[1], c.max_blocks)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda") if size else None
    pa.attention(c.pool, q, ints(slots), ints([n - 1 for n in lengths]), tables, out, workspace=ws)
    return out


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_evict_then_attend(kv):
    """Weights from the prompt's last rows and a decode row, the least looked-at
    keys dropped, pages given back: attention over what is left equals attention
    over exactly the kept tokens, and the freed pages are admitted again."""
    P, Hkv, G, D = 16, 2, 4, 128
    lengths, budget, window = [400, 250], 96, 32
    pages = pa.Pages(80, P, 4, 30)
    for i, n in enumerate(lengths):
        assert pages.admit(i, n, 20)[0] == pa.PA_OK
    free = pages.free_count()
    c = R.make_cache(lengths, Hkv=Hkv, D=D, P=P, kv=kv, seed=20, slots=[0, 1], spare_blocks=4)
    # the allocator's own tables, with the cache's contents behind them
    tables = torch.from_numpy(pages.block_tables).cuda()
    shape = (80, Hkv, P, D)
    k, v = (torch.zeros(shape, dtype=R.KV[kv], device="cuda") for _ in range(2))
    for i, n in enumerate(lengths):
        t = torch.arange(n, device="cuda")
        for new, old in ((k, c.k), (v, c.v)):
            new[tables[i][t // P].long(), :, t % P] = old[c.tables[i][t // P].long(), :, t % P]
    scale = np.asarray(c.scale.cpu()).reshape(-1) if kv == "e4m3" else 1.0
    c.pool, c.k, c.v, c.tables, c.max_blocks, c.num_seqs, c.max_tokens = pa.Pool(k, v, scale, scale), k, v, tables, 30, 4, 30 * P
    q = torch.randn(2 * window, Hkv * G, D, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).bfloat16()
    mass = torch.zeros(4, Hkv, c.max_tokens, device="cuda")
    seq = [i for i in range(2) for _ in range(window)]
    pos = [lengths[i] - window + j for i in range(2) for j in range(window)]
    chunks = [(0, window), (window, window)]
    size = pa.mass_workspace_bytes(c.pool, 2 * window, Hkv * G, 30, chunks)
    pa.attention_mass(c.pool, q, ints(seq), ints(pos), tables, mass, chunks=chunks,
                      workspace=torch.zeros(max(size, 1), dtype=torch.uint8, device="cuda"))
    keep = torch.empty(2, Hkv, budget, dtype=torch.int32, device="cuda")
    kept = torch.empty(2, dtype=torch.int32, device="cuda")
    pa.evict_select(mass, ints([0, 1]), ints(lengths), keep, kept_lengths=kept, keep_first=4, keep_last=16)
    old = [[R.cached(c, pool, i, n).clone() for i, n in enumerate(lengths)] for pool in (k, v)]
    before = mass.clone()
    pa.evict_compact(c.pool, keep, ints([0, 1]), ints(lengths), tables, mass=mass)
    torch.cuda.synchronize()
    assert kept.tolist() == [budget, budget]
    for i in range(2):
        pages.trim(i, budget + 20)
        for h in range(Hkv):
            at = keep[i, h].long()
            assert torch.equal(R.bits(R.cached(c, k, i, budget)[h]), R.bits(old[0][i][h, at]))
            assert torch.equal(mass[i, h, :budget], before[i, h, at])
            assert float(mass[i, h, budget:].abs().max()) == 0.0
    assert pages.free_count() == free + sum(-(-(n + 20) // P) - -(-(budget + 20) // P) for n in lengths)
    assert pages.admit(2, 300, 0)[0] == pa.PA_OK
    row = torch.randn(2, Hkv * G, D, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).bfloat16()
    out = attend(c, row, [0, 1], [budget, budget], torch.from_numpy(pages.block_tables).cuda())
    for i in range(2):
        kk = torch.stack([R.values(old[0][i][h, keep[i, h].long()]) for h in range(Hkv)]) * c.scale
        vv = torch.stack([R.values(old[1][i][h, keep[i, h].long()]) for h in range(Hkv)]) * c.scale
        s = torch.einsum("hgd,htd->hgt", row[i].double().view(Hkv, G, D), kk) / D ** 0.5
        ref = torch.einsum("hgt,htd->hgd", torch.softmax(s, dim=2), vv).reshape(Hkv * G, D)
        err = (out[i].double() - ref).abs()
        assert ((err <= 2e-3) | (err <= 1e-2 * ref.abs())).all()


def test_graph():
    """Selection and compaction captured together; replayed on new weights and lengths."""
    c = R.make_cache([300, 200], Hkv=2, D=64, P=16, seed=30)
    mass = torch.zeros(c.num_seqs, 2, c.max_tokens, device="cuda")
    lengths = ints([300, 200])
    keep = torch.empty(2, 2, 50, dtype=torch.int32, device="cuda")
    slots = ints(c.slots)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.evict_select(mass, slots, lengths, keep)
        pa.evict_compact(c.pool, keep, slots, lengths, c.tables, mass=mass)
    for seed, lens in ((1, [300, 200]), (2, [50, 49])):
        w = weights(mass.shape, "spread", seed).cuda()
        mass.copy_(w)
        lengths.copy_(ints(lens))
        old = [R.cached(c, c.k, s, n).clone() for s, n in zip(c.slots, lens)]
        graph.replay()
        torch.cuda.synchronize()
        for i, (s, n) in enumerate(zip(c.slots, lens)):
            for h in range(2):
                want = R.select_ref(w[s, h].cpu(), n, 50, 0, 0)
                assert keep[i, h, :len(want)].tolist() == want
                assert torch.equal(R.bits(R.cached(c, c.k, s, len(want))[h]), R.bits(old[i][h, want]))


@pytest.mark.parametrize("start", [0, 1999, 2001, 2500])
@pytest.mark.parametrize("copy", [False, True])
def test_compact_lists_out_of_order(start, copy):
    """A list that begins anew far down: what is not in order, or lies below its own place, is not moved;
    every other entry gets its own token's bytes and weight."""
    n, budget, turn = 6000, 3001, 2000
    c = R.make_cache([n, n] if copy else [n], Hkv=2, D=64, P=32, seed=6, slots=[0, 1] if copy else [0])
    j = torch.arange(budget)
    keep = torch.where(j < turn, 2999 + j, start + j - turn).to(torch.int32)
    before = torch.cat([torch.tensor([-1], dtype=torch.int32), keep[:-1]])
    moved = ((keep > before) & (keep >= j)).cuda()
    assert bool(moved[:turn].all()) and not bool(moved[turn])
    dst = 1 if copy else 0
    mass = torch.rand(c.num_seqs, 2, c.max_tokens, generator=torch.Generator().manual_seed(7)).cuda()
    old = [[R.cached(c, pool, s, n).clone() for s in (0, dst)] for pool in (c.k, c.v)]
    old_mass = mass.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.evict_compact(c.pool, keep.view(1, 1, -1).repeat(1, 2, 1).cuda(), ints([0]), ints([n]), c.tables, mass=mass,
                     dst_seq_ids=ints([dst]) if copy else None, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == pa.PA_ERR_OUT_OF_RANGE
    at = keep.long().cuda()
    for pool, (source, there) in zip((c.k, c.v), old):
        now = R.cached(c, pool, dst, n)
        want = there.clone()
        want[:, :budget] = torch.where(moved.view(1, -1, 1), source[:, at], there[:, :budget])
        assert torch.equal(R.bits(now), R.bits(want))
    want = torch.zeros_like(old_mass[0, :, :n])
    want[:, :budget] = torch.where(moved, old_mass[0][:, at], torch.zeros_like(old_mass[0][:, at]))
    assert torch.equal(mass[dst, :, :n], want)


def test_weights_that_change_during_the_call():
    """Another stream rewrites the weights while they are chosen from: which tokens come out is unspecified, but
    nothing is written outside the rows of the call."""
    n, T, budget = 32, 40000, 3000
    mass = weights((n, 4, T), "ties", 9).cuda()
    other = weights((n, 4, T), "spread", 10).cuda()
    room = torch.full((2 * n, 4, budget), -7, dtype=torch.int32, device="cuda")
    keep, slots, lengths = room[::2], ints(list(range(n))), ints([T] * n)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(30):
        with torch.cuda.stream(side):
            for _ in range(4):
                mass.copy_(other)
                mass.mul_(0.5).round_()
        for k in range(n):  # a row of `room` each, with untouched ones between
            pa.evict_select(mass, slots[k:k + 1], lengths[k:k + 1], keep[k:k + 1], keep_first=4, keep_last=64)
    torch.cuda.synchronize()
    assert (room[1::2] == -7).all()
    assert ((keep == -7) | ((keep >= 0) & (keep < T))).all()  # (or not written)
