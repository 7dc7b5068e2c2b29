"""pa_attention_mass over chunks of the types that run on warp-level MMAs (f32
and e4m3 pools, f32 queries) against a 64-bit reference: several key ranges and
key blocks, many columns, every head group, refused and poisoned rows."""
import pytest
import torch

import cache_ref as R
from test_gpu_mass import check, queries, run

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
KINDS = [("e4m3", BF16), ("e4m3", F32), ("bf16", F32), ("f32", BF16), ("f32", F32)]


def every_kind(f):
    return pytest.mark.parametrize("D", [64, 128])(pytest.mark.parametrize("kv,q_dtype", KINDS)(f))


def zeros(c):
    return torch.zeros(c.num_seqs, c.Hkv, c.max_tokens, device="cuda")


@every_kind
@pytest.mark.parametrize("rows,length,G,P", [(64, 5000, 4, 16), (33, 2049, 8, 64), (7, 3100, 5, 256)])
def test_long_windows(kv, q_dtype, D, rows, length, G, P):
    """The last rows of a prompt of several key ranges; per-head scales where the pool is e4m3."""
    c = R.make_cache([length], Hkv=2, D=D, P=P, kv=kv, seed=length)
    q = queries(rows, 2 * G, D, q_dtype, seed=length)
    check(c, q, c.slots * rows, [length - rows + i for i in range(rows)], [(0, rows)])


@every_kind
@pytest.mark.parametrize("rows,start,G", [(1300, 0, 1), (301, 2100, 5), (513, 1, 8)])
def test_long_chunks(kv, q_dtype, D, rows, start, G):
    """Whole prompts and long parts: keys that the first blocks of columns do not see."""
    c = R.make_cache([start + rows], Hkv=1, D=D, P=32, kv=kv, seed=rows)
    q = queries(rows, G, D, q_dtype, seed=rows)
    check(c, q, c.slots * rows, list(range(start, start + rows)), [(0, rows)])


@every_kind
@pytest.mark.parametrize("rows", [1, 2, 17])
def test_short_chunks_beside_rows(kv, q_dtype, D, rows):
    """Sixteen chunks, the most a call takes, with decode rows between them."""
    lengths = [rows + 131 * i for i in range(16)] + [700, 1]
    c = R.make_cache(lengths, Hkv=2, D=D, P=16, kv=kv, seed=rows)
    seq, pos, chunks = [], [], []
    for i in range(16):
        if i in (3, 9):
            k = 16 + i // 9
            seq.append(c.slots[k])
            pos.append(lengths[k] - 1)
        chunks.append((len(seq), rows))
        seq += [c.slots[i]] * rows
        pos += [lengths[i] - rows + r for r in range(rows)]
    check(c, queries(len(seq), 6, D, q_dtype, seed=rows), seq, pos, chunks)


@every_kind
def test_bits_do_not_depend_on_the_batch(kv, q_dtype, D):
    rows = 150
    c = R.make_cache([2900, 1333, 700 + rows], Hkv=2, D=D, P=16, kv=kv, seed=13)
    q = queries(3 * rows, 6, D, q_dtype, seed=13)
    seq = [s for s in c.slots for _ in range(rows)]
    pos = [n - rows + i for n in c.lengths for i in range(rows)]
    whole = zeros(c)
    assert run(c, q, seq, pos, whole, [(i * rows, rows) for i in range(3)]) == 0
    for i, s in enumerate(c.slots):
        one, part = zeros(c), slice(i * rows, (i + 1) * rows)
        assert run(c, q[part].contiguous(), seq[part], pos[part], one, [(0, rows)]) == 0
        assert torch.equal(one[s], whole[s])


@every_kind
@pytest.mark.parametrize("rows", [20, 130])
def test_nan_query_stays_with_the_keys_it_sees(kv, q_dtype, D, rows):
    c = R.make_cache([1700], Hkv=2, D=D, P=32, kv=kv, seed=16)
    q = queries(rows, 6, D, q_dtype)
    clean, mass, s = zeros(c), zeros(c), c.slots[0]
    pos = [1700 - rows + i for i in range(rows)]
    assert run(c, q, c.slots * rows, pos, clean, [(0, rows)]) == 0
    q[7] = float("nan")
    assert run(c, q, c.slots * rows, pos, mass, [(0, rows)]) == 0
    assert torch.isnan(mass[s, :, :pos[7] + 1]).all()
    assert torch.equal(mass[s, :, pos[7] + 1:], clean[s, :, pos[7] + 1:])


@pytest.mark.parametrize("kv,q_dtype", KINDS)
@pytest.mark.parametrize("what", ["sequence", "negative", "position", "page", "another sequence", "a gap"])
def test_bad_chunks_add_nothing(kv, q_dtype, what):
    rows = 20
    c = R.make_cache([100, 120], Hkv=2, D=64, P=16, kv=kv, seed=12)
    seq = [c.slots[0]] * rows + [c.slots[1]]
    pos = [100 - rows + i for i in range(rows)] + [119]
    q = queries(rows + 1, 4, 64, q_dtype)
    tables, good = c.tables.clone(), zeros(c)
    assert run(c, q[rows:].contiguous(), seq[rows:], pos[rows:], good) == 0
    if what == "sequence":
        seq[:rows] = [c.num_seqs] * rows
    elif what == "negative":
        seq[:rows] = [-1] * rows
    elif what == "position":
        pos[:rows] = [c.max_tokens - rows + 1 + i for i in range(rows)]
    elif what == "page":
        tables[c.slots[0], 2] = c.k.shape[0]
    elif what == "another sequence":
        seq[5] = c.slots[1]
    else:
        pos[5] += 1
    mass = zeros(c)
    assert run(c, q, seq, pos, mass, [(0, rows)], tables=tables) == 3  # out of range
    assert torch.equal(mass, good)
