"""The cache operators on pages whose offsets pass 32 bits: the same calls on a
small pool and on a large one that holds its pages at the far end, bit for bit."""
import pytest
import torch

import cache_ref as R
import paged_kv_continuous_pa_gb300 as pa

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module", params=["bf16", "e4m3"])
def far(request):
    """(small, large): caches of the same contents; the large pool has 2^32 elements and more."""
    c = R.make_cache([1500, 1500, 700], Hkv=8, D=128, P=256, kv=request.param, seed=1, spare_blocks=2)
    n = c.k.shape[0]
    pages = (1 << 32) // (8 * 256 * 128) + n
    pools = [torch.empty((pages,) + c.k.shape[1:], dtype=c.k.dtype, device="cuda") for _ in range(2)]
    scale = c.scale.view(-1).cpu().float().numpy() if c.kv == "e4m3" else 1.0
    handle = pa.Pool(*pools, scale, scale)
    yield c, handle, pools, pages - n
    del handle, pools
    torch.cuda.empty_cache()


def both(far):
    """Fresh copies of the small cache, one of them at the far end: (pool, k, v, tables) each."""
    c, handle, pools, base = far
    small = [c.k.clone(), c.v.clone()]
    scale = c.scale.view(-1).cpu().float().numpy() if c.kv == "e4m3" else 1.0
    for big, x in zip(pools, small):
        big[base:].copy_(x)
    return [(pa.Pool(*small, scale, scale), *small, c.tables.clone()),
            (handle, pools[0][base:], pools[1][base:], c.tables + base)]


@pytest.mark.parametrize("q_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows", [1, 40])
def test_mass(far, q_dtype, rows):
    c = far[0]
    q = torch.randn(2 * rows, 16, 128, generator=torch.Generator().manual_seed(2)).to(q_dtype).cuda()
    seq = [s for s in c.slots[:2] for _ in range(rows)]
    pos = [1500 - rows + i for i in range(rows)] * 2
    chunks = [(0, rows), (rows, rows)] if rows > 1 else []
    got = []
    for pool, _, _, tables in both(far):
        mass = torch.zeros(c.num_seqs, c.Hkv, c.max_tokens, device="cuda")
        size = pa.mass_workspace_bytes(pool, 2 * rows, 16, c.max_blocks, chunks)
        status = ints([0])
        pa.attention_mass(pool, q, ints(seq), ints(pos), tables, mass, chunks=chunks, status=status,
                          workspace=torch.empty(max(size, 1), dtype=torch.uint8, device="cuda"))
        assert int(status.item()) == 0
        got.append(mass)
    assert float(got[0].sum()) > 0 and torch.equal(got[0], got[1])


def test_compact(far):
    c = far[0]
    g = torch.Generator().manual_seed(3)
    keep = torch.stack([torch.stack([torch.randperm(1500, generator=g)[:600].sort().values for _ in range(8)]) for _ in range(2)])
    got = []
    for pool, k, v, tables in both(far):
        status = ints([0])
        pa.evict_compact(pool, keep.to(torch.int32).cuda(), ints(c.slots[:2]), ints([1500, 1500]), tables,
                         dst_seq_ids=ints([c.slots[0], c.slots[2]]), status=status)
        assert int(status.item()) == 0
        got.append((R.bits(k).clone(), R.bits(v).clone()))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert not torch.equal(got[0][0], R.bits(c.k))


def test_reorder(far):
    c, base = far[0], far[3]
    got = []
    for i, (pool, k, v, tables) in enumerate(both(far)):
        status = ints([0])
        pa.beam_reorder(pool, ints([[1, 0]]), ints([c.slots[:2]]), ints([1500]), tables, status=status)
        assert int(status.item()) == 0
        got.append((R.bits(k).clone(), R.bits(v).clone(), tables - i * base))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert not torch.equal(got[0][0], R.bits(c.k))


def test_rows_of_sums_beyond_32_bits():
    """Weights of a slot whose row starts behind 2^32 elements of the buffer: added, chosen and moved there."""
    c = R.make_cache([900], Hkv=4, D=64, P=256, seed=4, slots=[0])
    blocks = 1 << 14
    slots = (1 << 32) // (4 * blocks * 256) + 2
    tables = torch.full((slots, blocks), -1, dtype=torch.int32, device="cuda")
    tables[slots - 1, :c.max_blocks] = c.tables[0]
    mass = torch.empty(slots, 4, blocks * 256, device="cuda")
    mass[slots - 1].zero_()
    q = torch.randn(1, 8, 64, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    status = ints([0])
    pa.attention_mass(c.pool, q, ints([slots - 1]), ints([899]), tables, mass, status=status)
    want, big = R.mass_of_rows(c, q, [0], [899])
    got = mass[slots - 1, :, :c.max_tokens].double()
    bound = R.mass_bound(c, want[0], torch.zeros_like(want[0]), big, 1, 2)
    assert ((got - want[0]).abs() <= bound).all()
    keep = torch.empty(1, 4, 100, dtype=torch.int32, device="cuda")
    pa.evict_select(mass, ints([slots - 1]), ints([900]), keep, status=status)
    before = mass[slots - 1].clone()
    for h in range(4):
        assert keep[0, h].tolist() == R.select_ref(before[h].cpu(), 900, 100, 0, 0)
    old = R.cached(c, c.k, 0, 900).clone()
    pa.evict_compact(c.pool, keep, ints([slots - 1]), ints([900]), tables, mass=mass, status=status)
    assert int(status.item()) == 0
    for h in range(4):
        at = keep[0, h].long()
        assert torch.equal(mass[slots - 1, h, :100], before[h, at])
        assert torch.equal(R.bits(R.cached(c, c.k, 0, 100)[h]), R.bits(old[h, at]))
