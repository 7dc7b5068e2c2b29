"""pa_attention_mass against a 64-bit reference: types, head groups, page and
sequence lengths, chunks (observation windows and whole prompts), strangers'
memory, refused rows, streams and graphs."""
import pytest
import torch

import cache_ref as R
import paged_kv_continuous_pa_gb300 as pa

pytestmark = pytest.mark.gpu


def run(c, q, seq_ids, positions, mass, chunks=(), **kw):
    ids = torch.tensor(seq_ids, dtype=torch.int32, device="cuda")
    pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
    size = pa.mass_workspace_bytes(c.pool, len(seq_ids), q.shape[1], c.max_blocks, chunks)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xA5) if size else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.attention_mass(c.pool, q, ids, pos, kw.pop("tables", c.tables), mass, chunks=chunks, workspace=ws, status=status,
                      **kw)
    torch.cuda.synchronize()
    return int(status.item())


def check(c, q, seq_ids, positions, chunks=(), seed=0, **kw):
    g = torch.Generator().manual_seed(100 + seed)
    before = (torch.rand(c.num_seqs, c.Hkv, c.max_tokens, generator=g) * 3).cuda()
    mass = before.clone()
    assert run(c, q, seq_ids, positions, mass, chunks, **kw) == 0
    added, big = R.mass_of_rows(c, q, seq_ids, positions, kw.get("softmax_scale"))
    rows = max([1] + [n for _, n in chunks])
    bound = R.mass_bound(c, added, before.double(), big, rows, q.shape[1] // c.Hkv)
    err = (mass.double() - before.double() - added).abs()
    assert torch.isfinite(mass).all()
    assert (err <= bound).all(), f"worst {float((err / bound).max()):.3g} of the bound"
    touched = torch.zeros_like(mass, dtype=torch.bool)
    for s, p in zip(seq_ids, positions):
        touched[s, :, :p + 1] = True
    assert torch.equal(mass[~touched], before[~touched])
    return mass


def queries(n, hq, d, dtype, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(7 + seed)
    return (torch.randn(n, hq, d, generator=g) * scale).to(dtype).cuda()


@pytest.mark.parametrize("kv", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("q_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
def test_types(kv, q_dtype, D):
    c = R.make_cache([1, 15, 16, 17, 300, 1029], Hkv=2, D=D, P=16, kv=kv, seed=1)
    q = queries(6, 6, D, q_dtype)
    check(c, q, c.slots, [n - 1 for n in c.lengths])


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("kv,q_dtype", [("bf16", torch.bfloat16), ("e4m3", torch.float32)])
def test_groups(G, kv, q_dtype):
    c = R.make_cache([33, 700], Hkv=3, D=128, P=32, kv=kv, seed=G)
    q = queries(2, 3 * G, 128, q_dtype, seed=G)
    check(c, q, c.slots, [n - 1 for n in c.lengths])


@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("window", [1, 40])
def test_page_sizes(P, window):
    c = R.make_cache([P - 1 + window, P + window, 5 * P + 3 + window], Hkv=2, D=64, P=P, seed=P)
    n = len(c.lengths)
    q = queries(n * window, 4, 64, torch.bfloat16, seed=P)
    seq = [s for s in c.slots for _ in range(window)]
    pos = [x - window + i for x in c.lengths for i in range(window)]
    check(c, q, seq, pos, [(i * window, window) for i in range(n)] if window > 1 else ())


@pytest.mark.parametrize("length", [4095, 4097, 9001, 33000])
@pytest.mark.parametrize("G", [2, 8])
def test_long_rows(length, G):
    c = R.make_cache([length, 5], Hkv=1, D=128, P=64, seed=length)
    q = queries(2, G, 128, torch.bfloat16, seed=length)
    check(c, q, c.slots, [length - 1, 4])


def test_very_long_row():
    """More keys than one cluster keeps scores for."""
    c = R.make_cache([150001], Hkv=1, D=64, P=256, seed=3)
    q = queries(1, 8, 64, torch.bfloat16)
    check(c, q, c.slots, [150000])


def test_rows_that_look_back():
    """A row may sit before the end of its cache: later keys stay untouched."""
    c = R.make_cache([200, 300], Hkv=2, D=64, P=32, seed=5)
    q = queries(2, 4, 64, torch.bfloat16)
    check(c, q, c.slots, [0, 31])


@pytest.mark.parametrize("softmax_scale", [0.02, 1.0])
def test_scales(softmax_scale):
    c = R.make_cache([257], Hkv=2, D=64, P=16, seed=6)
    check(c, queries(1, 4, 64, torch.bfloat16), c.slots, [256], softmax_scale=softmax_scale)


@pytest.mark.parametrize("rows", [2, 15, 16, 17, 40, 129, 300])
@pytest.mark.parametrize("G", [1, 3, 4, 8])
def test_chunks(rows, G):
    """Windows at the end of a prompt, whole prompts (start 0), and decode rows beside them."""
    c = R.make_cache([rows, rows + 77, 50, 4000], Hkv=2, D=128, P=32, seed=rows + G)
    seq = [c.slots[0]] * rows + [c.slots[2]] + [c.slots[1]] * rows + [c.slots[3]]
    pos = list(range(rows)) + [49] + [77 + i for i in range(rows)] + [3999]
    q = queries(len(seq), 2 * G, 128, torch.bfloat16, seed=rows)
    check(c, q, seq, pos, [(0, rows), (rows + 1, rows)])


@pytest.mark.parametrize("D,P,length", [(64, 16, 5000), (128, 256, 4600), (128, 16, 9000)])
def test_long_windows(D, P, length):
    rows = 64
    c = R.make_cache([length], Hkv=2, D=D, P=P, seed=length)
    q = queries(rows, 8, D, torch.bfloat16)
    check(c, q, c.slots * rows, [length - rows + i for i in range(rows)], [(0, rows)])


@pytest.mark.parametrize("kv,q_dtype", [("e4m3", torch.bfloat16), ("f32", torch.bfloat16), ("bf16", torch.float32)])
def test_chunks_of_other_types(kv, q_dtype):
    rows = 21
    c = R.make_cache([90, 30], Hkv=2, D=64, P=16, kv=kv, seed=8)
    seq = [c.slots[0]] * rows + [c.slots[1]]
    pos = [90 - rows + i for i in range(rows)] + [29]
    check(c, queries(rows + 1, 6, 64, q_dtype), seq, pos, [(0, rows)])


def test_large_scores():
    """Scores far apart: one key takes all the weight, the others vanish."""
    c = R.make_cache([500], Hkv=1, D=64, P=16, seed=9)
    q = queries(1, 2, 64, torch.bfloat16, scale=30.0)
    check(c, q, c.slots, [499])


def test_bits_do_not_depend_on_the_batch():
    c = R.make_cache([900, 64, 2000, 333, 2001, 17], Hkv=2, D=128, P=32, seed=10)
    q = queries(6, 8, 128, torch.bfloat16)
    pos = [n - 1 for n in c.lengths]
    whole = torch.zeros(c.num_seqs, c.Hkv, c.max_tokens, device="cuda")
    assert run(c, q, c.slots, pos, whole) == 0
    for i in range(6):
        one = torch.zeros_like(whole)
        assert run(c, q[i:i + 1].contiguous(), c.slots[i:i + 1], pos[i:i + 1], one) == 0
        assert torch.equal(one[c.slots[i]], whole[c.slots[i]])
    again = torch.zeros_like(whole)
    assert run(c, q, c.slots, pos, again) == 0
    assert torch.equal(again, whole)


def test_chunk_bits_do_not_depend_on_the_batch():
    rows = 40
    c = R.make_cache([900, 700], Hkv=2, D=128, P=32, seed=11)
    q = queries(2 * rows, 4, 128, torch.bfloat16)
    seq = [c.slots[0]] * rows + [c.slots[1]] * rows
    pos = [900 - rows + i for i in range(rows)] + [700 - rows + i for i in range(rows)]
    whole = torch.zeros(c.num_seqs, c.Hkv, c.max_tokens, device="cuda")
    assert run(c, q, seq, pos, whole, [(0, rows), (rows, rows)]) == 0
    one = torch.zeros_like(whole)
    assert run(c, q[rows:].contiguous(), seq[rows:], pos[rows:], one, [(0, rows)]) == 0
    assert torch.equal(one[c.slots[1]], whole[c.slots[1]])


@pytest.mark.parametrize("what", ["sequence", "negative", "position", "page"])
@pytest.mark.parametrize("rows", [1, 20])
def test_bad_rows_add_nothing(what, rows):
    """A bad row (or a tile-path chunk with one) is reported; the others are as without it."""
    c = R.make_cache([100, 120], Hkv=2, D=64, P=16, seed=12)
    seq = [c.slots[0]] * rows + [c.slots[1]]
    pos = [100 - rows + i for i in range(rows)] + [119]
    q = queries(rows + 1, 4, 64, torch.bfloat16)
    chunks = [(0, rows)] if rows > 1 else ()
    tables = c.tables
    good = torch.zeros(c.num_seqs, c.Hkv, c.max_tokens, device="cuda")
    assert run(c, q[rows:].contiguous(), seq[rows:], pos[rows:], good) == 0
    if what == "sequence":
        seq = [c.num_seqs] * rows + seq[rows:]
    elif what == "negative":
        seq = [-1] * rows + seq[rows:]
    elif what == "position":
        pos = [c.max_tokens - rows + 1 + i for i in range(rows)] + pos[rows:]
    else:
        tables = tables.clone()
        tables[c.slots[0], 2] = c.k.shape[0]
    mass = torch.zeros_like(good)
    assert run(c, q, seq, pos, mass, chunks, tables=tables) == pa.PA_ERR_OUT_OF_RANGE
    assert torch.equal(mass, good)


def test_poison_beside_the_queries():
    """Rows behind a chunk and other chunks' rows never leak in (NaN queries beside it)."""
    rows = 50
    c = R.make_cache([400, 300], Hkv=2, D=128, P=32, seed=13)
    q = queries(rows + 1, 6, 128, torch.bfloat16)
    q[rows:] = float("nan")
    seq, pos = [c.slots[0]] * rows + [c.slots[1]], [400 - rows + i for i in range(rows)] + [299]
    mass = torch.zeros(c.num_seqs, c.Hkv, c.max_tokens, device="cuda")
    assert run(c, q, seq, pos, mass, [(0, rows)]) == 0
    clean = torch.zeros_like(mass)
    assert run(c, q[:rows].contiguous(), seq[:rows], pos[:rows], clean, [(0, rows)]) == 0
    assert torch.isfinite(mass[c.slots[0]]).all()
    assert torch.equal(mass[c.slots[0]], clean[c.slots[0]])


def test_no_rows():
    c = R.make_cache([10], Hkv=2, D=64, P=16)
    mass = torch.ones(c.num_seqs, c.Hkv, c.max_tokens, device="cuda")
    pa.attention_mass(c.pool, torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda"),
                      torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"),
                      c.tables, mass)
    assert torch.equal(mass, torch.ones_like(mass))


def test_stream_and_graph():
    """On a stream of its own, captured and replayed: each replay adds the same weights."""
    rows = 32
    c = R.make_cache([600, 500], Hkv=2, D=128, P=32, seed=14)
    seq, pos = [c.slots[0]] * rows + [c.slots[1]], [600 - rows + i for i in range(rows)] + [499]
    q = queries(rows + 1, 4, 128, torch.bfloat16)
    ids = torch.tensor(seq, dtype=torch.int32, device="cuda")
    positions = torch.tensor(pos, dtype=torch.int32, device="cuda")
    chunks = [(0, rows)]
    size = pa.mass_workspace_bytes(c.pool, rows + 1, 4, c.max_blocks, chunks)
    ws = torch.zeros(max(size, 1), dtype=torch.uint8, device="cuda")
    mass = torch.zeros(c.num_seqs, c.Hkv, c.max_tokens, device="cuda")
    want = torch.zeros_like(mass)
    assert run(c, q, seq, pos, want, chunks) == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pa.attention_mass(c.pool, q, ids, positions, c.tables, mass, chunks=chunks, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(mass, want)
    graph.replay()
    torch.cuda.synchronize()
    # the buffer is rounded at most once for each row that adds to it: on the second replay a
    # half step (2^-24) of a sum no larger than the final one, and as much on the first
    assert ((mass - 2 * want).abs() <= 2 * rows * 2.0 ** -24 * 2 * want).all()


def test_matches_the_attention_step():
    """With V the unit vectors of each key, the attention's output is the weights."""
    c = R.make_cache([60], Hkv=1, D=64, P=64, kv="f32", seed=15, spare_blocks=0)
    page = int(c.tables[c.slots[0], 0])
    c.v.zero_()
    c.v[page, 0] = torch.eye(64, device="cuda")
    q = queries(1, 4, 64, torch.float32)
    ids = torch.tensor(c.slots, dtype=torch.int32, device="cuda")
    pos = torch.tensor([59], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    pa.attention(c.pool, q, ids, pos, c.tables, out)
    mass = torch.zeros(c.num_seqs, 1, 64, device="cuda")
    pa.attention_mass(c.pool, q, ids, pos, c.tables, mass)
    # two FP32 evaluations of the same weights, each within (64 + 8) roundings of scores below 8
    assert torch.allclose(mass[c.slots[0], 0, :60], out[0].sum(dim=0)[:60], rtol=2 * 72 * 2.0 ** -23 * 8 * 2, atol=1e-7)


@pytest.mark.parametrize("rows", [20, 130])
def test_nan_query_stays_with_the_keys_it_sees(rows):
    """One row of a chunk has a NaN query: the keys behind its position are as if it were not there."""
    c = R.make_cache([700], Hkv=2, D=128, P=32, seed=16)
    q = queries(rows, 6, 128, torch.bfloat16)
    clean = torch.zeros(c.num_seqs, c.Hkv, c.max_tokens, device="cuda")
    pos = [700 - rows + i for i in range(rows)]
    assert run(c, q, c.slots * rows, pos, clean, [(0, rows)]) == 0
    bad = 7
    q[bad] = float("nan")
    mass = torch.zeros_like(clean)
    assert run(c, q, c.slots * rows, pos, mass, [(0, rows)]) == 0
    s = c.slots[0]
    assert torch.isnan(mass[s, :, :pos[bad] + 1]).all()
    # the rows that see the keys behind it are the same ones: the same weights
    assert torch.equal(mass[s, :, pos[bad] + 1:700], clean[s, :, pos[bad] + 1:700])


def test_wait_limit_runs_out_cleanly():
    """The tile path's bounded waits: with the injected stall the call reports PA_ERR_TIMEOUT, adds nothing,
    and the next call is right."""
    rows = 32
    c = R.make_cache([600], Hkv=2, D=128, P=32, seed=17)
    q = queries(rows, 4, 128, torch.bfloat16)
    seq, pos = c.slots * rows, [600 - rows + i for i in range(rows)]
    mass = torch.zeros(c.num_seqs, c.Hkv, c.max_tokens, device="cuda")
    pa.set_wait_limit(1000)
    pa.debug_stall_waits(True)
    try:
        assert run(c, q, seq, pos, mass, [(0, rows)]) == pa.PA_ERR_TIMEOUT
    finally:
        pa.debug_stall_waits(False)
        pa.set_wait_limit(0)
    assert torch.equal(mass, torch.zeros_like(mass))
    check(c, q, seq, pos, [(0, rows)])


@pytest.mark.parametrize("rows,start,G", [(2500, 0, 1), (1300, 900, 2), (700, 5000, 3), (513, 1, 8)])
def test_long_chunks(rows, start, G):
    """Many column tiles over several key ranges: every pair of tiles, with ranges and tiles that see only part."""
    c = R.make_cache([start + rows], Hkv=1, D=64, P=32, seed=rows)
    q = queries(rows, G, 64, torch.bfloat16, seed=rows)
    check(c, q, c.slots * rows, list(range(start, start + rows)), [(0, rows)])


def test_many_short_units():
    """More pieces of work than CTAs, some of one key tile, so that a CTA's warps reach its next piece at
    different times: right, and the same bits each time."""
    lengths = [1030 + 37 * i for i in range(12)]
    c = R.make_cache(lengths, Hkv=32, D=64, P=16, seed=41)
    q = queries(16 * 12, 32, 64, torch.bfloat16, seed=41)
    seq = [s for s in c.slots for _ in range(16)]
    pos = [n - 16 + i for n in c.lengths for i in range(16)]
    chunks = [(16 * i, 16) for i in range(12)]
    first = check(c, q, seq, pos, chunks, seed=41)
    for _ in range(5):
        assert torch.equal(check(c, q, seq, pos, chunks, seed=41), first)


@pytest.mark.parametrize("G", [1, 4])
def test_long_chunk_bits_do_not_depend_on_the_batch(G):
    """Several column tiles to a key, and more pieces of work than CTAs before the chunk's own."""
    rows = 500
    c = R.make_cache([2900, 2333, 700 + rows], Hkv=8, D=64, P=16, seed=13)
    q = queries(3 * rows, 8 * G, 64, torch.bfloat16, seed=13)
    seq = [s for s in c.slots for _ in range(rows)]
    pos = [n - rows + i for n in c.lengths for i in range(rows)]
    whole = torch.zeros(c.num_seqs, c.Hkv, c.max_tokens, device="cuda")
    assert run(c, q, seq, pos, whole, [(i * rows, rows) for i in range(3)]) == 0
    for i, s in enumerate(c.slots):
        one = torch.zeros_like(whole)
        part = slice(i * rows, (i + 1) * rows)
        assert run(c, q[part].contiguous(), seq[part], pos[part], one, [(0, rows)]) == 0
        assert torch.equal(one[s], whole[s])


@pytest.mark.parametrize("kv,q_dtype,D", [("f32", torch.float32, 128), ("e4m3", torch.bfloat16, 64), ("bf16", torch.float32, 128)])
def test_wide_tables(kv, q_dtype, D):
    """Tables of more than 2^16 tokens take the largest clusters, whatever the rows' own lengths."""
    c = R.make_cache([66001, 1, 300], Hkv=1, D=D, P=256, kv=kv, seed=17)
    check(c, queries(3, 8, D, q_dtype, seed=17), c.slots, [66000, 0, 299])


@pytest.mark.parametrize("rows", [1, 2, 7])
@pytest.mark.parametrize("G", [1, 5])
def test_short_chunks(rows, G):
    c = R.make_cache([rows, 1500 + rows, 4100], Hkv=2, D=128, P=16, seed=19)
    q = queries(3 * rows, 2 * G, 128, torch.bfloat16, seed=19)
    seq = [s for s in c.slots for _ in range(rows)]
    pos = [n - rows + i for n in c.lengths for i in range(rows)]
    check(c, q, seq, pos, [(i * rows, rows) for i in range(3)])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_two_calls_at_once(kv):
    """Two streams, two workspaces, two sums: the bits of the calls one after the other."""
    rows = 64
    c = R.make_cache([3000, 2500, 1800], Hkv=4, D=128, P=32, kv=kv, seed=23)
    seq = torch.tensor([s for s in c.slots for _ in range(rows)], dtype=torch.int32, device="cuda")
    pos = torch.tensor([n - rows + i for n in c.lengths for i in range(rows)], dtype=torch.int32, device="cuda")
    chunks = [(i * rows, rows) for i in range(3)]
    q = [queries(3 * rows, 16, 128, torch.bfloat16, seed=s) for s in (23, 24)]
    size = pa.mass_workspace_bytes(c.pool, 3 * rows, 16, c.max_blocks, chunks)
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in q]
    streams = [torch.cuda.Stream() for _ in q]
    mass = torch.zeros(2, 2, c.num_seqs, c.Hkv, c.max_tokens, device="cuda")  # [one by one | at once][query]
    for i in range(2):
        pa.attention_mass(c.pool, q[i], seq, pos, c.tables, mass[0, i], chunks=chunks, workspace=ws[i])
        torch.cuda.synchronize()
    for _ in range(4):
        mass[1].zero_()
        torch.cuda.synchronize()
        for i in range(2):
            pa.attention_mass(c.pool, q[i], seq, pos, c.tables, mass[1, i], chunks=chunks, workspace=ws[i], stream=streams[i])
        torch.cuda.synchronize()
        assert torch.equal(mass[0], mass[1])


# ------------------------------------------- infinities, and values beside them --

def set_key(c, t, h, d, value):
    c.k[c.tables[c.slots[0], t // c.P].long(), h, t % c.P, d] = value


def window(length, rows):
    """Positions of the last rows of a sequence, and its chunks (none for one row)."""
    return [length - rows + i for i in range(rows)], [(0, rows)] if rows > 1 else []


def check_against(c, q, pos, chunks, big):
    """The added weights against 64 bits, `big` as in mass_bound; NaN where the reference has it."""
    rows = len(pos)
    before = torch.rand(c.num_seqs, c.Hkv, c.max_tokens, generator=torch.Generator().manual_seed(3)).cuda()
    mass = before.clone()
    assert run(c, q, c.slots * rows, pos, mass, chunks) == 0
    added, _ = R.mass_of_rows(c, q, c.slots * rows, pos)
    assert torch.equal(torch.isnan(mass), torch.isnan(added))
    bound = R.mass_bound(c, added, before.double(), big, rows, q.shape[1] // c.Hkv)
    err = (mass.double() - before.double() - added).abs()
    assert ((err <= bound) | torch.isnan(added)).all()
    return mass, before


TYPES = [("f32", torch.float32), ("f32", torch.bfloat16), ("bf16", torch.float32), ("bf16", torch.bfloat16)]


@pytest.mark.parametrize("kv,q_dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [1, 40])
def test_infinite_keys(kv, q_dtype, D, rows):
    """A key whose score is -infinity gets no weight, and the others theirs."""
    c = R.make_cache([1700], Hkv=2, D=D, P=16, kv=kv, seed=31)
    q = queries(rows, 6, D, q_dtype, seed=31)
    q[:, :, 5] = q[:, :, 5].abs() + 0.1
    q[:, :, D - 3] = -q[:, :, D - 3].abs() - 0.1
    q[0, :, 5] = 0.5  # nothing of it is left behind the leading bits
    pos, chunks = window(1700, rows)
    _, big = R.mass_of_rows(c, q, c.slots * rows, pos)
    none = [(0, 0), (0, 3), (0, 8), (1, 17), (1, 1023), (0, 1024), (1, 1699)]
    for i, (h, t) in enumerate(none):
        set_key(c, t, h, 5, float("-inf")) if i % 2 else set_key(c, t, h, D - 3, float("inf"))
    mass, before = check_against(c, q, pos, chunks, big)
    assert torch.isfinite(mass).all()
    for h, t in none:
        assert float(mass[c.slots[0], h, t]) == float(before[c.slots[0], h, t])


@pytest.mark.parametrize("kv,q_dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 40])
def test_infinite_scores(kv, q_dtype, rows):
    """A score of +infinity leaves no weights to the rows that see the key; other rows and heads keep theirs."""
    c = R.make_cache([1700], Hkv=2, D=64, P=16, kv=kv, seed=32)
    q = queries(rows, 4, 64, q_dtype, seed=32)
    q[:, :, 5] = q[:, :, 5].abs() + 0.1
    pos, chunks = window(1700, rows)
    _, big = R.mass_of_rows(c, q, c.slots * rows, pos)
    set_key(c, 1690, 1, 5, float("inf"))
    mass, _ = check_against(c, q, pos, chunks, big)
    s = c.slots[0]
    assert torch.isnan(mass[s, 1, :1700]).all() and torch.isfinite(mass[s, 0]).all()


@pytest.mark.parametrize("kv,q_dtype,large", [("f32", torch.float32, "key"), ("f32", torch.bfloat16, "key"),
                                              ("f32", torch.float32, "query"), ("bf16", torch.float32, "query")])
@pytest.mark.parametrize("rows", [1, 40])
def test_largest_values(kv, q_dtype, large, rows):
    """f32 values above the largest bf16 one, against ones that bring the product back."""
    c = R.make_cache([300], Hkv=2, D=64, P=16, kv=kv, seed=33)
    q = queries(rows, 4, 64, q_dtype, seed=33)
    most, least = 3.4e38, 2e-38
    for h in range(2):
        for t in range(300):
            set_key(c, t, h, 5, (most if t % 3 else -most) if large == "key" else (least if t % 3 else -least))
    q[:, :, 5] = least if large == "key" else most
    pos, chunks = window(300, rows)
    _, big = R.mass_of_rows(c, q, c.slots * rows, pos)
    mass, _ = check_against(c, q, pos, chunks, big)
    assert torch.isfinite(mass).all()


@pytest.mark.parametrize("kv,q_dtype", TYPES)
@pytest.mark.parametrize("length", [4000, 9001])
def test_infinite_keys_in_long_rows(kv, q_dtype, length):
    """More scores than a CTA keeps, or a cluster of CTAs."""
    c = R.make_cache([length], Hkv=1, D=64, P=16, kv=kv, seed=34)
    q = queries(1, 8, 64, q_dtype, seed=34)
    q[:, :, 5] = q[:, :, 5].abs() + 0.1
    _, big = R.mass_of_rows(c, q, c.slots, [length - 1])
    for t in (1, 2500, 3500, 3999, length - 1):
        set_key(c, t, 0, 5, float("-inf"))
    mass, before = check_against(c, q, [length - 1], [], big)
    assert torch.isfinite(mass).all() and float(mass[c.slots[0], 0, 3500]) == float(before[c.slots[0], 0, 3500])


@pytest.mark.parametrize("kv,q_dtype", TYPES + [("e4m3", torch.bfloat16), ("e4m3", torch.float32)])
@pytest.mark.parametrize("scale", [1e2, 1e4, 1e6, 1e9, 1e20, 1e34])
@pytest.mark.parametrize("rows,length,start", [(1, 1700, None), (1, 1700, 0), (40, 40, 0), (40, 2500, 0), (300, 2500, 0)])
def test_weights_sum_to_one_at_any_score(kv, q_dtype, scale, rows, length, start):
    """A row's weights are a distribution however large its finite scores are (start None: outside the chunks)."""
    c = R.make_cache([length], Hkv=2, D=128, P=16, kv=kv, seed=36)
    q = queries(rows, 8, 128, q_dtype, seed=36, scale=scale)
    pos, _ = window(length, rows)
    mass = torch.zeros(c.num_seqs, c.Hkv, c.max_tokens, device="cuda")
    assert run(c, q, c.slots * rows, pos, mass, [] if start is None else [(0, rows)]) == 0
    # a column's statistics against its weights: 2^-14 ln 2 at most (twice half a step of scores up to 1024 in the
    # log2 domain; larger ones are taken relative to their maximum), ex2.approx 2^-22 twice, FP32 sums of at most
    # `length` weights and rows * 4 columns, half a step 2^-24 an addition
    tol = 2.0 ** -14 * 0.6932 + 2.0 ** -21 + (length + rows * 4) * 2.0 ** -24
    total = mass[c.slots[0]].double().sum(dim=1)
    assert ((total - rows * 4).abs() <= tol * rows * 4).all(), (total / (rows * 4)).tolist()
    assert float(mass.max()) <= rows * 4 * (1 + tol)
