"""The 4-bit cache: append, read and attention against 64-bit references; steps, strangers'
memory, refused rows, streams and graphs; pa_read_kv over every pool type."""
import pytest
import torch

import cache_ref as C
import paged_kv_continuous_pa_gb300 as pa
import serving_ref as R

pytestmark = pytest.mark.gpu


class Cache4:
    """A 4-bit pool whose slots outside the sequences hold NaN ranges; pages in random order."""

    def __init__(self, lengths, hkv=2, d=64, page=16, seed=0, spare=1):
        g = torch.Generator().manual_seed(seed)
        n = len(lengths)
        self.seqs, self.blocks = n + 2, max(1, max(-(-x // page) for x in lengths) + spare)
        self.slots, self.lengths = torch.randperm(self.seqs, generator=g)[:n].tolist(), list(lengths)
        pages = self.seqs * self.blocks
        order = torch.randperm(pages, generator=g).view(self.seqs, self.blocks)
        self.hkv, self.d, self.page = hkv, d, page
        self.codes = [torch.randint(0, 256, (pages, hkv, page, d // 2), generator=g, dtype=torch.uint8) for _ in "kv"]
        self.ranges = []
        for _ in "kv":
            pair = torch.full((pages, hkv, page, 2), float("nan"), dtype=torch.float16)
            for slot, length in zip(self.slots, lengths):
                t = torch.arange(length)
                step = torch.rand(length, hkv, generator=g) * 0.3 + 0.1
                low = -step * (torch.rand(length, hkv, generator=g) * 5 + 5)
                pair[order[slot][t // page], :, t % page] = torch.stack([step, low], dim=2).half()
            self.ranges.append(pair)
        self.codes, self.ranges = [x.cuda() for x in self.codes], [x.cuda() for x in self.ranges]
        self.tables = order.to(torch.int32).cuda()
        self.pool = pa.Pool(*self.codes, k_ranges=self.ranges[0], v_ranges=self.ranges[1])

    def cached(self, side, slot, length):
        """(float64 values [Hkv, length, D], ranges [Hkv, length, 2])"""
        t = torch.arange(length, device="cuda")
        at = self.tables[slot][t // self.page].long()
        codes, pair = (x[side][at, :, t % self.page].transpose(0, 1) for x in (self.codes, self.ranges))
        return R.values4(codes, pair), pair


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def queries(n, hq, d, dtype, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(7 + seed)
    return (torch.randn(n, hq, d, generator=g) * scale).to(dtype).cuda()


def attend(c, q, seqs, positions, chunks=(), **kw):
    out = torch.full_like(q, 7.0)
    size = pa.workspace_bytes(c.pool, len(seqs), q.shape[1], c.blocks, chunks)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda") if size else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.attention(c.pool, q, ints(seqs), ints(positions), c.tables, out, chunks=chunks, workspace=ws, status=status, **kw)
    torch.cuda.synchronize()
    return out, int(status.item())


def check(c, q, seqs, positions, chunks=(), softmax_scale=None):
    out, status = attend(c, q, seqs, positions, chunks, softmax_scale=softmax_scale or 0.0)
    assert status == 0
    compare(c, q, seqs, positions, out, softmax_scale)
    return out


def compare(c, q, seqs, positions, out, softmax_scale=None):
    scale = softmax_scale or R.scale_of(c.d)
    for r, (s, p) in enumerate(zip(seqs, positions)):
        (k, kr), (v, vr) = c.cached(0, s, p + 1), c.cached(1, s, p + 1)
        want, weights = R.attend4(q[r], k, v, scale)
        bound = R.attend4_bound(q[r], want, weights, kr, vr, scale)
        err = (out[r].double() - want).abs()
        assert (err <= bound).all(), f"row {r} at {p}: {float((err / bound).max()):.3g} of the bound"


@pytest.mark.parametrize("q_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
def test_lengths(q_dtype, d):
    c = Cache4([1, 15, 16, 17, 31, 32, 33, 127, 300, 1029], d=d, seed=1)
    check(c, queries(10, 6, d, q_dtype), c.slots, [n - 1 for n in c.lengths])


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("q_dtype", [torch.bfloat16, torch.float32])
def test_groups(G, q_dtype):
    c = Cache4([33, 700], hkv=3, d=128, page=32, seed=G)
    check(c, queries(2, 3 * G, 128, q_dtype, seed=G), c.slots, [32, 699])


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_sizes(page):
    c = Cache4([page - 1, page, page + 1, 5 * page + 3], d=64, page=page, seed=page)
    check(c, queries(4, 4, 64, torch.bfloat16), c.slots, [n - 1 for n in c.lengths])


@pytest.mark.parametrize("q_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("length", [4096, 4097, 20011])
def test_long_rows(length, q_dtype):
    """Splits, and sums of many small weights."""
    c = Cache4([length, 5], hkv=1, d=128, page=64, seed=length)
    check(c, queries(2, 5, 128, q_dtype, scale=0.2), c.slots, [length - 1, 4])


def test_short_splits():
    c = Cache4([1000, 70], hkv=2, d=64, page=256, seed=3)
    old = pa.get_split_tokens()
    pa.set_split_tokens(64)
    try:
        check(c, queries(2, 8, 64, torch.bfloat16), c.slots, [999, 69])
    finally:
        pa.set_split_tokens(old)


def test_rows_that_look_back():
    c = Cache4([200, 300], seed=5)
    check(c, queries(2, 4, 64, torch.bfloat16), c.slots, [0, 31])


@pytest.mark.parametrize("softmax_scale", [0.02, 2.0])
def test_scales(softmax_scale):
    c = Cache4([257], seed=6)
    check(c, queries(1, 4, 64, torch.bfloat16), c.slots, [256], softmax_scale=softmax_scale)


def test_chunk_rows_and_order():
    """Chunks run row by row; the launch order and the company change no bits."""
    c = Cache4([40 + (i * 97) % 1500 for i in range(150)], hkv=2, d=64, page=16, seed=7)
    seqs = c.slots + [c.slots[0]] * 20
    pos = [n - 1 for n in c.lengths] + [c.lengths[0] - 20 + i for i in range(20)]
    seqs, pos = seqs[1:], pos[1:]  # the chunk's sequence is in it alone
    q = queries(len(seqs), 4, 64, torch.bfloat16)
    out = check(c, q, seqs, pos, [(len(seqs) - 20, 20)])
    old = pa.get_unit_order()
    try:
        for mode in (pa.PA_ORDER_CALL, pa.PA_ORDER_LONGEST_FIRST):
            pa.set_unit_order(mode)
            assert torch.equal(attend(c, q, seqs, pos, [(len(seqs) - 20, 20)])[0], out)
    finally:
        pa.set_unit_order(old)
    for r in (0, 17, len(seqs) - 1):
        assert torch.equal(attend(c, q[r:r + 1].contiguous(), seqs[r:r + 1], pos[r:r + 1])[0], out[r:r + 1])


def test_noalloc():
    c = Cache4([5000, 77], hkv=2, d=128, page=64, seed=8)
    q = queries(2, 4, 128, torch.bfloat16)
    want = check(c, q, c.slots, [4999, 76])
    out = torch.empty_like(q)
    pa.attention_noalloc(c.pool, q, ints(c.slots), ints([4999, 76]), c.tables, out)
    assert torch.equal(out, want)


def test_nan_range_reaches_its_reader_alone():
    c = Cache4([100, 100], hkv=2, d=64, page=16, seed=9)
    q = queries(2, 4, 64, torch.bfloat16)
    clean, _ = attend(c, q, c.slots, [99, 99])
    at = int(c.tables[c.slots[0], 60 // 16])
    c.ranges[1][at, 1, 60 % 16] = float("nan")
    out, status = attend(c, q, c.slots, [99, 99])
    assert status == 0
    assert torch.isnan(out[0, 2:]).all()
    assert torch.equal(out[0, :2], clean[0, :2]) and torch.equal(out[1], clean[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 32)])
def test_append_and_read(dtype, d, page):
    """Codes and ranges as the format's steps give them, bit for bit; other slots as they were."""
    c = Cache4([0, 0, 0], hkv=3, d=d, page=page, seed=2, spare=5)
    g = torch.Generator().manual_seed(3)
    seqs, pos = [], []
    for slot, first, n in zip(c.slots, (0, page - 1, 2 * page + 3), (1, 40, 17)):
        seqs += [slot] * n
        pos += list(range(first, first + n))
    n = len(seqs)
    size = 10.0 ** (torch.rand(n, 3, 1, generator=g) * 8 - 5)
    new = [(torch.randn(n, 3, d, generator=g) * size + size * torch.randn(n, 3, 1, generator=g)).to(dtype) for _ in "kv"]
    new[0][0] = 3.25  # no range
    new[0][1] = 0.0
    new[1][2, 0] = 1e-9  # a range that f16 does not hold
    new[1][3, 1, 5] = float("inf")
    new[1][3, 1, 6] = -1e30
    new[0][4, 2, 7] = float("nan")
    new = [x.cuda() for x in new]
    want_codes, want_ranges = [x.clone() for x in c.codes], [x.clone() for x in c.ranges]
    at = c.tables[torch.tensor(seqs).cuda(), torch.tensor(pos).cuda() // page].long()
    slot = torch.tensor(pos).cuda() % page
    for side in (0, 1):
        code, step, low = (x.cuda() for x in R.encode4(new[side].cpu()))
        want_codes[side][at, :, slot] = R.pack4(code)
        want_ranges[side][at, :, slot] = torch.cat([step, low], dim=2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.append_kv(c.pool, new[0], new[1], ints(seqs), ints(pos), c.tables, status=status)
    for side in (0, 1):
        assert torch.equal(c.codes[side], want_codes[side])
        fine = ~torch.isnan(want_ranges[side])
        assert torch.equal(torch.isnan(c.ranges[side]), ~fine)
        assert torch.equal(c.ranges[side][fine], want_ranges[side][fine])
    for out_dtype in (torch.float32, torch.bfloat16):
        k, v = (torch.zeros(n, 3, d, dtype=out_dtype, device="cuda") for _ in "kv")
        pa.read_kv(c.pool, ints(seqs), ints(pos), c.tables, k, v, status=status)
        for side, got in ((0, k), (1, v)):
            want = R.values4(want_codes[side][at, :, slot], want_ranges[side][at, :, slot]).float().to(out_dtype)
            fine = ~torch.isnan(want)
            assert torch.equal(torch.isnan(got), ~fine) and torch.equal(got[fine], want[fine])
        alone = torch.zeros_like(v)
        pa.read_kv(c.pool, ints(seqs), ints(pos), c.tables, v_out=alone)
        assert torch.equal(alone.nan_to_num(), v.nan_to_num())
    assert int(status.item()) == 0
    # half a step at most (and the roundings of the range), where nothing was clamped
    for side in (0, 1):
        x = new[side].double()
        ok = torch.isfinite(x).all(dim=2, keepdim=True) & (x.abs().amax(dim=2, keepdim=True) < 6e4)
        y = R.values4(want_codes[side][at, :, slot], want_ranges[side][at, :, slot])
        step = want_ranges[side][at, :, slot][..., :1].double()
        slack = step * (0.5 + 15 * 2.0 ** -11) + x.abs().amax(dim=2, keepdim=True) * 2.0 ** -11 + 2.0 ** -20
        assert ((y - x).abs() <= slack)[ok.expand_as(x)].all()


def test_step_is_append_then_attention():
    lengths = [40, 300, 5000, 17]
    a, b = (Cache4(lengths, hkv=2, d=128, page=16, seed=4) for _ in "ab")
    seqs = a.slots[:3] + [a.slots[3]] * 6
    pos = [n for n in lengths[:3]] + [17 + i for i in range(6)]
    chunks = [(3, 6)]
    q = queries(9, 8, 128, torch.bfloat16)
    k, v = queries(9, 2, 128, torch.bfloat16, seed=1), queries(9, 2, 128, torch.bfloat16, seed=2)
    pa.append_kv(a.pool, k, v, ints(seqs), ints(pos), a.tables)
    want = check(a, q, seqs, pos, chunks)
    out = torch.empty_like(q)
    ws = torch.zeros(pa.workspace_bytes(b.pool, 9, 8, b.blocks, chunks), dtype=torch.uint8, device="cuda")
    for mode in (pa.PA_ORDER_AUTO, pa.PA_ORDER_LONGEST_FIRST):
        old = pa.get_unit_order()
        pa.set_unit_order(mode)
        try:
            ws = torch.zeros(pa.workspace_bytes(b.pool, 9, 8, b.blocks, chunks), dtype=torch.uint8, device="cuda")
            pa.step(b.pool, q, k, v, ints(seqs), ints(pos), b.tables, out, chunks=chunks, workspace=ws)
            torch.cuda.synchronize()
        finally:
            pa.set_unit_order(old)
        assert torch.equal(out, want)
        for side in (0, 1):
            assert torch.equal(a.codes[side], b.codes[side])
            assert torch.equal(C.bits(a.ranges[side]), C.bits(b.ranges[side]))


def test_bad_rows():
    """A bad row gets zeros and an error; its neighbours are right."""
    c = Cache4([50, 60, 70], seed=11)
    q = queries(4, 4, 64, torch.bfloat16)
    seqs, pos = [c.slots[0], c.seqs + 3, c.slots[1], -1], [49, 5, 59, 0]
    out, status = attend(c, q, seqs, pos)
    assert status == pa.PA_ERR_OUT_OF_RANGE and (out[[1, 3]] == 0).all()
    compare(c, q[[0, 2]], [seqs[0], seqs[2]], [49, 59], out[[0, 2]])
    tables = c.tables.clone()
    c.tables[c.slots[2], 1] = c.seqs * c.blocks
    out, status = attend(c, q[:2].contiguous(), [c.slots[0], c.slots[2]], [49, 69])
    assert status == pa.PA_ERR_OUT_OF_RANGE and (out[1] == 0).all()
    # append and read skip such rows
    k, v = queries(2, 2, 64, torch.bfloat16, seed=1), queries(2, 2, 64, torch.bfloat16, seed=2)
    before = [x.clone() for x in c.codes]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.append_kv(c.pool, k, v, ints([c.slots[2], 99]), ints([20, 0]), c.tables, status=status)
    assert int(status.item()) == pa.PA_ERR_OUT_OF_RANGE and all(torch.equal(x, y) for x, y in zip(before, c.codes))
    status.zero_()
    ko = torch.ones(3, 2, 64, device="cuda")
    pa.read_kv(c.pool, ints([c.slots[2], 99, c.slots[0]]), ints([20, 0, 3]), c.tables, k_out=ko, status=status)
    assert int(status.item()) == pa.PA_ERR_OUT_OF_RANGE and (ko[:2] == 0).all()
    c.tables = tables
    assert torch.equal(ko[2].double(), c.cached(0, c.slots[0], 4)[0][:, 3].float().double())


def test_far_pages():
    """Pages whose byte offsets pass 32 bits."""
    hkv, d, page = 8, 128, 256
    pages = 2 ** 32 // (hkv * page * d // 2) + 40
    codes = [torch.zeros(pages, hkv, page, d // 2, dtype=torch.uint8, device="cuda") for _ in "kv"]
    ranges = [torch.zeros(pages, hkv, page, 2, dtype=torch.float16, device="cuda") for _ in "kv"]
    c = Cache4.__new__(Cache4)
    c.hkv, c.d, c.page, c.seqs, c.blocks, c.codes, c.ranges = hkv, d, page, 2, 2, codes, ranges
    c.tables = ints([[pages - 1, 3], [pages - 30, pages - 7]])
    c.pool = pa.Pool(*codes, k_ranges=ranges[0], v_ranges=ranges[1])
    seqs, pos = [0] * 300 + [1] * 500, list(range(300)) + list(range(500))
    k, v = queries(800, hkv, d, torch.bfloat16, seed=1), queries(800, hkv, d, torch.bfloat16, seed=2)
    pa.append_kv(c.pool, k, v, ints(seqs), ints(pos), c.tables)
    check(c, queries(2, 16, d, torch.bfloat16), [0, 1], [299, 499])
    out = torch.empty(800, hkv, d, device="cuda")
    pa.read_kv(c.pool, ints(seqs), ints(pos), c.tables, v_out=out)
    assert torch.equal(out[300:].double(), c.cached(1, 1, 500)[0].transpose(0, 1).float().double())


def test_wait_that_runs_out():
    c = Cache4([300], seed=1)
    q = queries(1, 4, 64, torch.bfloat16)
    pa.set_wait_limit(2000)
    pa.debug_stall_waits(True)
    try:
        _, status = attend(c, q, c.slots, [299])
    finally:
        pa.debug_stall_waits(False)
        pa.set_wait_limit(0)
    assert status == pa.PA_ERR_TIMEOUT
    check(c, q, c.slots, [299])


def test_graph():
    """A captured step; positions and inputs change between replays."""
    c = Cache4([100, 3000], hkv=2, d=64, page=32, seed=2)
    q, k, v = (queries(2, h, 64, torch.bfloat16, seed=h) for h in (8, 2, 2))
    ids, pos = ints(c.slots), ints([100, 3000])
    out = torch.zeros_like(q)
    ws = torch.zeros(max(1, pa.workspace_bytes(c.pool, 2, 8, c.blocks)), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pa.step(c.pool, q, k, v, ids, pos, c.tables, out, workspace=ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pa.step(c.pool, q, k, v, ids, pos, c.tables, out, workspace=ws)
    for i in range(3):
        pos.copy_(ints([100 + i, 3000 + i]))
        q.copy_(queries(2, 8, 64, torch.bfloat16, seed=20 + i))
        k.copy_(queries(2, 2, 64, torch.bfloat16, seed=30 + i))
        graph.replay()
        torch.cuda.synchronize()
        compare(c, q, c.slots, [100 + i, 3000 + i], out)


@pytest.mark.parametrize("kv", ["f32", "bf16", "e4m3"])
def test_read_other_pools(kv):
    c = C.make_cache([70, 33], Hkv=2, D=64, P=16, kv=kv, seed=3)
    seqs, pos = [c.slots[0]] * 70 + [c.slots[1]] * 33 + [c.slots[0]], list(range(70)) + list(range(33)) + [5]
    for dtype in (torch.float32, torch.bfloat16):
        k, v = (torch.zeros(104, 2, 64, dtype=dtype, device="cuda") for _ in "kv")
        pa.read_kv(c.pool, ints(seqs), ints(pos), c.tables, k, v)
        for got, pool in ((k, c.k), (v, c.v)):
            want = torch.cat([C.values(C.cached(c, pool, c.slots[i], n), c.scale).transpose(0, 1) for i, n in ((0, 70), (1, 33))])
            want = torch.cat([want, want[5:6]]).float().to(dtype)
            assert torch.equal(got, want)


def test_calls_that_do_not_take_it():
    c = Cache4([20], seed=1)
    q = queries(1, 2, 64, torch.bfloat16)
    mass = torch.zeros(c.seqs, 2, c.blocks * 16, device="cuda")
    for call in (lambda: pa.attention_mass(c.pool, q, ints(c.slots), ints([19]), c.tables, mass),
                 lambda: pa.evict_compact(c.pool, torch.zeros(1, 2, 4, dtype=torch.int32, device="cuda"), ints(c.slots), ints([20]), c.tables),
                 lambda: pa.beam_reorder(c.pool, ints([[0]]), ints([c.slots]), ints([20]), c.tables)):
        with pytest.raises(pa.PaError) as e:
            call()
        assert e.value.status == pa.PA_ERR_UNSUPPORTED


@pytest.mark.parametrize("length", [8, 53, 700])
@pytest.mark.parametrize("d", [64, 128])
def test_f32_rows_lose_nothing_to_the_codes_offset(d, length):
    """Norm of the error against the norm of the result.  With centred codes partial sums of scores stay below 4 (log2
    domain, queries and values of size 1, scale 1 / sqrt(D)); their 16 or fewer truncations of 2^-23 and the weights' own
    2^-21 make weights off by 2^-17 at most, most of it in common, which a softmax divides out; sums of weights times centred values are
    of the result's own size.  2^-17 of the norm in all; sums over codes 0..15 are 8 sqrt(length) times as large
    beside their result and truncated as often, 2^-16 and more at 53 keys."""
    c = Cache4([length] * 16, hkv=4, d=d, page=32, seed=length)
    q = queries(16, 16, d, torch.float32, seed=d)
    out = attend(c, q, c.slots, [length - 1] * 16)
    out = out[0] if isinstance(out, tuple) else out
    want = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for i, slot in enumerate(c.slots):
        k, v = c.cached(0, slot, length)[0], c.cached(1, slot, length)[0]
        want[i] = R.attend4(q[i], k, v, R.scale_of(d))[0]
    err = float((out.double() - want).norm() / want.norm())
    assert err <= 2.0 ** -17, err
