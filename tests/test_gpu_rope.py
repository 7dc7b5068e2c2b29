"""Rotary positions against a 64-bit reference: layouts, parts of a head, scalings, far
positions, pool types, packed rows, in place, the transposed map as gradient, bad rows, graphs."""
import math

import pytest
import torch

import cache_ref as C
import paged_kv_continuous_pa_gb300 as pa
import serving_ref as R

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def normal(shape, dtype, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def frequencies(rot, base=10000.0):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


def assert_rotated(got, x, positions, rope, rot, interleaved, inverse=False):
    f, m = rope.frequencies()
    want, size = R.rotate(x, positions, f, m, rot, interleaved, inverse)
    err = (got.double() - want).abs()
    bound = R.rotate_bound(size, want, got.dtype)
    assert (err <= bound).all(), f"{float((err / bound).max()):.3g} of the bound"
    assert torch.equal(got[:, :, rot:], x[:, :, rot:])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (64, 64), (64, 16), (64, 2), (128, 20), (128, 126), (64, 34)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows(layout, d, rot, dtype):
    x = normal((9, 5, d), dtype, rot)
    positions = ints([0, 1, 2, 77, 4095, 131071, 1000003, 2 ** 31 - 1, -12345])
    rope = pa.Rope(rot, layout=layout)
    out = torch.zeros_like(x)
    pa.rope_rows(rope, x, positions, out)
    assert_rotated(out, x, positions, rope, rot, layout == "interleaved")
    back = torch.zeros_like(x)
    pa.rope_rows(rope, x, positions, back, inverse=True)
    assert_rotated(back, x, positions, rope, rot, layout == "interleaved", inverse=True)
    same = x.clone()
    pa.rope_rows(rope, same, positions)
    assert torch.equal(same, out)


@pytest.mark.parametrize("n", [1, 700, 1025, 4097, 9001])
def test_row_counts(n):
    x = normal((n, 3, 64), torch.bfloat16, n)
    positions = torch.randint(0, 100000, (n,), dtype=torch.int32, device="cuda")
    rope = pa.Rope(64)
    out = torch.zeros_like(x)
    pa.rope_rows(rope, x, positions, out)
    assert_rotated(out, x, positions, rope, 64, False)


def test_scalings():
    """The frequencies by their definitions."""
    rot, factor, length = 64, 8.0, 4096
    f = frequencies(rot)
    got, m = pa.Rope(rot).frequencies()
    assert got.tolist() == pytest.approx(f, rel=1e-14) and m == 1.0
    got, m = pa.Rope(rot, scaling="linear", factor=factor).frequencies()
    assert got.tolist() == pytest.approx([x / factor for x in f], rel=1e-14) and m == 1.0
    got, m = pa.Rope(rot, scaling="base", factor=factor).frequencies()
    assert got.tolist() == pytest.approx(frequencies(rot, 10000.0 * factor ** (rot / (rot - 2))), rel=1e-13)
    # the slowest pair of a changed base is the slowest one of the linear scaling
    assert got[-1] == pytest.approx(f[-1] / factor, rel=1e-12)
    got, m = pa.Rope(rot, scaling="ramp", factor=factor, original_positions=length).frequencies()
    at = [rot * math.log(length / (2 * math.pi * t)) / (2 * math.log(10000.0)) for t in (32.0, 1.0)]
    lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
    want = [x * (1 - w) + x / factor * w for i, x in enumerate(f) for w in [min(max((i - lo) / (hi - lo), 0), 1)]]
    assert got.tolist() == pytest.approx(want, rel=1e-13) and m == pytest.approx(0.1 * math.log(factor) + 1, rel=1e-14)
    assert got[0] == pytest.approx(f[0]) and got[-1] == pytest.approx(f[-1] / factor)
    got, m = pa.Rope(rot, scaling="bands", factor=factor, original_positions=length, magnitude=0.5).frequencies()
    want = [x * w + x / factor * (1 - w) for x in f for w in [min(max((length * x / (2 * math.pi) - 1) / 3, 0), 1)]]
    assert got.tolist() == pytest.approx(want, rel=1e-13) and m == 0.5


def make_pool(kv, seqs, blocks, hkv, d, page, seed=0):
    """A pool filled with noise, pages in random order; the 4-bit kind too."""
    g = torch.Generator().manual_seed(seed)
    pages = seqs * blocks
    tables = torch.randperm(pages, generator=g).view(seqs, blocks).to(torch.int32).cuda()
    if kv == "int4":
        codes = [torch.randint(0, 256, (pages, hkv, page, d // 2), generator=g, dtype=torch.uint8).cuda() for _ in "kv"]
        ranges = [torch.rand(pages, hkv, page, 2, generator=g).half().cuda() for _ in "kv"]
        return pa.Pool(*codes, k_ranges=ranges[0], v_ranges=ranges[1]), tables, codes + ranges
    pools = [C.random_rows((pages, hkv, page, d), kv, g).cuda() for _ in "kv"]
    return pa.Pool(*pools, *((0.03, 0.05) if kv == "e4m3" else ())), tables, pools


@pytest.mark.parametrize("kv", ["f32", "bf16", "e4m3", "int4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout,d,rot", [("half", 128, 128), ("interleaved", 64, 32), ("half", 64, 20)])
def test_append(kv, dtype, layout, d, rot):
    """Queries as rope_rows gives them, keys within the rotation's bound of the stored form's
    rounding, values as append_kv stores them, other slots untouched."""
    n, hq, hkv, page, seqs, blocks = 45, 6, 2, 16, 4, 9
    qkv = normal((n, hq + 2 * hkv, d), dtype, 5)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    ids = ints([0] * 20 + [2] * 25)
    pos = ints(list(range(5, 25)) + list(range(100, 125)))
    rope = pa.Rope(rot, layout=layout, scaling="linear", factor=4.0, magnitude=1.25)
    pool, tables, held = make_pool(kv, seqs, blocks, hkv, d, page, 1)
    before = [x.clone() for x in held]
    q_out, status = torch.zeros(n, hq, d, dtype=dtype, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.rope_append(pool, rope, q, k, v, ids, pos, tables, q_out, status=status)
    assert int(status.item()) == 0
    assert_rotated(q_out, q, pos, rope, rot, layout == "interleaved")
    f, m = rope.frequencies()
    want, size = R.rotate(k, pos, f, m, rot, layout == "interleaved")
    ko, vo = (torch.zeros(n, hkv, d, device="cuda") for _ in "kv")
    pa.read_kv(pool, ids, pos, tables, ko, vo)
    err, wide = (ko.double() - want).abs(), want.abs() + 2.0 ** -21 * size
    if kv == "f32":
        step = 2.0 ** -24 * wide
    elif kv == "bf16":
        step = 2.0 ** -8 * wide
    elif kv == "e4m3":  # half a step, 2^-4 of a normal and 2^-10 scales of a subnormal value; codes end at 448
        step = torch.maximum(2.0 ** -4 * wide, torch.full_like(wide, 2.0 ** -10 * 0.03))
    else:  # half a step of the row's own range, whose two numbers are f16
        span = want.amax(dim=2, keepdim=True) - want.amin(dim=2, keepdim=True)
        step = span / 15 * (0.5 + 2.0 ** -6) + 2.0 ** -10 * wide.amax(dim=2, keepdim=True)
    assert (err <= step + 2.0 ** -20 * size).all()
    # values, and everything else in the pool, as an append of the values alone leaves them
    other, _, held2 = make_pool(kv, seqs, blocks, hkv, d, page, 1)
    pa.append_kv(other, k.contiguous(), v.contiguous(), ids, pos, tables)
    vo2 = torch.zeros_like(vo)
    pa.read_kv(other, ids, pos, tables, v_out=vo2)
    assert torch.equal(vo, vo2)
    mine = torch.zeros(held[0].shape[0], page, dtype=torch.bool, device="cuda")
    mine[tables[ids.long(), pos.long() // page].long(), pos.long() % page] = True
    for x, y in zip(held, before):
        assert torch.equal(C.bits(x.transpose(1, 2)[~mine]), C.bits(y.transpose(1, 2)[~mine]))


@pytest.mark.parametrize("kv", ["f32", "bf16", "e4m3", "int4"])
def test_append_without_rotation(kv):
    """rope None: the bytes that append_kv stores; no queries."""
    n, hkv, d, page = 30, 3, 64, 32
    k, v = normal((n, hkv, d), torch.bfloat16, 1), normal((n, hkv, d), torch.bfloat16, 2)
    k[3, 1, 5], v[4, 0, 0] = float("nan"), float("inf")
    ids, pos = ints([1] * n), ints(list(range(n)))
    a, tables, held_a = make_pool(kv, 2, 2, hkv, d, page)
    b, _, held_b = make_pool(kv, 2, 2, hkv, d, page)
    pa.rope_append(a, None, None, k, v, ids, pos, tables, None)
    pa.append_kv(b, k, v, ids, pos, tables)
    for x, y in zip(held_a, held_b):
        assert torch.equal(C.bits(x), C.bits(y))


def test_in_place_and_bad_rows():
    n, hq, hkv, d, page = 12, 4, 2, 128, 16
    q, k, v = (normal((n, h, d), torch.bfloat16, h) for h in (hq, hkv, 3))
    v = v[:, :hkv].contiguous()
    pool, tables, held = make_pool("bf16", 3, 3, hkv, d, page)
    tables[2, 1] = 9  # no such page
    ids, pos = ints([0, 0, 7, 1, -1, 1, 2, 2, 0, 0, 1, 1]), ints([0, 1, 2, 0, 3, 47, 15, 16, -1, 48, 5, 6])
    bad = torch.tensor([2, 4, 7, 8, 9], device="cuda")
    good = torch.tensor([0, 1, 3, 5, 6, 10, 11], device="cuda")
    rope = pa.Rope(128)
    before, x, status = [y.clone() for y in held], q.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.rope_append(pool, rope, x, k, v, ids, pos, tables, x, status=status)
    assert int(status.item()) == pa.PA_ERR_OUT_OF_RANGE
    assert torch.equal(x[bad], q[bad])
    assert_rotated(x[good], q[good], pos[good], rope, 128, False)
    at, slot = tables[ids[good].long(), pos[good].long() // page].long(), pos[good].long() % page
    before[1][at, :, slot] = v[good]
    before[0][at, :, slot] = held[0][at, :, slot]
    assert torch.equal(held[1], before[1]) and torch.equal(held[0], before[0])


def test_gradient():
    """The transposed map gives the gradient of the formula, and of differences."""
    x = normal((4, 2, 64), torch.float32, 1)
    positions = ints([3, 500, 70000, 11])
    rope = pa.Rope(48, layout="half", magnitude=1.5)
    f, m = rope.frequencies()
    go = normal((4, 2, 64), torch.float32, 2)
    grad = torch.zeros_like(x)
    pa.rope_rows(rope, go, positions, grad, inverse=True)
    leaf = x.double().requires_grad_()
    angle = positions.double().view(-1, 1, 1) * torch.as_tensor(f, device="cuda")
    c, s = angle.cos() * m, angle.sin() * m
    a, b = leaf[:, :, :24], leaf[:, :, 24:48]
    torch.cat([a * c - b * s, a * s + b * c, leaf[:, :, 48:]], dim=2).backward(go.double())
    assert ((grad.double() - leaf.grad).abs() <= R.rotate_bound(4 * m * torch.ones_like(leaf), leaf.grad, x.dtype)).all()
    # the map is linear: its change along e is its value at e
    e = normal((4, 2, 64), torch.float32, 3)
    out = torch.zeros_like(x)
    pa.rope_rows(rope, e, positions, out)
    left, right = (out.double() * go.double()).sum(), (e.double() * grad.double()).sum()
    assert abs(left - right) <= 2.0 ** -20 * (out.double().abs() * go.double().abs()).sum() * 4


def test_graph():
    q, k, v = (normal((8, h, 64), torch.bfloat16, h) for h in (4, 2, 1))
    v = v.expand(8, 2, 64).contiguous()
    pool, tables, held = make_pool("bf16", 8, 4, 2, 64, 16)
    ids, pos = ints(list(range(8))), ints([5] * 8)
    rope, q_out = pa.Rope(64), torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pa.rope_append(pool, rope, q, k, v, ids, pos, tables, q_out)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pa.rope_append(pool, rope, q, k, v, ids, pos, tables, q_out)
    pos.copy_(ints(list(range(20, 28))))
    graph.replay()
    torch.cuda.synchronize()
    assert_rotated(q_out, q, pos, rope, 64, False)
