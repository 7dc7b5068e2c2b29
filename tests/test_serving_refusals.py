"""What the serving operators (tables, rotary positions, prompt attention, the 4-bit pool and
reads) refuse, at the C ABI and in the binding.  Nothing here launches: every call fails a host-side check or
has nothing to do."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_continuous_pa_gb300 as pa
from paged_kv_continuous_pa_gb300 import build as pa_build

VP = ctypes.c_void_p
DEV = VP(0x100000)   # any address: no call here reads it
ODD = VP(0x100004)
BAD, NO, OK = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED, pa.PA_OK


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return pa.load()


def pool_desc(**kw):
    d = dict(num_pages=16, page_size=32, num_kv_heads=2, head_dim=64, kv_dtype=pa.PA_INT4, k_scale=1.0, v_scale=1.0)
    d.update(kw)
    return pa.PoolDesc(**d)


def create_int4(lib, desc, kc=0x10000, vc=0x20000, kr=0x30000, vr=0x40000):
    h = VP()
    return lib.pa_pool_create_int4(ctypes.byref(desc) if desc is not None else None, VP(kc), VP(vc), VP(kr), VP(vr), ctypes.byref(h)), h


@pytest.fixture(scope="module")
def pool(lib):
    st, h = create_int4(lib, pool_desc())
    assert st == OK
    yield h
    lib.pa_pool_destroy(h)


def rope_desc(**kw):
    d = dict(rotary_dim=64, layout=0, base=10000.0, scaling=0, factor=1.0, original_positions=0, low=0.0, high=0.0, magnitude=0.0)
    d.update(kw)
    return pa.RopeDesc(**d)


def create_rope(lib, **kw):
    h = VP()
    return lib.pa_rope_create(ctypes.byref(rope_desc(**kw)), ctypes.byref(h)), h


@pytest.fixture(scope="module")
def rope(lib):
    st, h = create_rope(lib)
    assert st == OK
    yield h
    lib.pa_rope_destroy(h)


# ------------------------------------------------------------------------------------ the pool --
def test_int4_pool_sizes(lib):
    d = pool_desc()
    assert lib.pa_pool_bytes(ctypes.byref(d)) == 16 * 2 * 32 * 64 // 2
    assert lib.pa_pool_range_bytes(ctypes.byref(d)) == 16 * 2 * 32 * 4
    assert lib.pa_pool_range_bytes(ctypes.byref(pool_desc(kv_dtype=pa.PA_BF16))) == 0
    assert lib.pa_pool_range_bytes(None) == 0
    far = pool_desc(num_pages=1 << 24, page_size=256, num_kv_heads=8, head_dim=128)
    assert lib.pa_pool_bytes(ctypes.byref(far)) == (1 << 24) * 8 * 256 * 64
    assert lib.pa_pool_range_bytes(ctypes.byref(far)) == (1 << 24) * 8 * 256 * 4


@pytest.mark.parametrize("kw,want", [
    (dict(kv_dtype=pa.PA_BF16), BAD), (dict(head_dim=96), NO), (dict(page_size=48), NO), (dict(page_size=8), NO),
    (dict(num_pages=0), BAD), (dict(num_kv_heads=0), BAD)])
def test_int4_pool_descriptions(lib, kw, want):
    assert create_int4(lib, pool_desc(**kw))[0] == want


@pytest.mark.parametrize("name", ["kc", "vc", "kr", "vr"])
@pytest.mark.parametrize("address", [0, 0x10008])
def test_int4_pool_addresses(lib, name, address):
    assert create_int4(lib, pool_desc(), **{name: address})[0] == BAD


def test_int4_pool_other_refusals(lib, pool):
    assert create_int4(lib, None)[0] == BAD
    h = VP()
    assert lib.pa_pool_create(ctypes.byref(pool_desc()), VP(0x10000), VP(0x20000), ctypes.byref(h)) == BAD
    assert lib.pa_pool_create_int4(ctypes.byref(pool_desc()), VP(0x10000), VP(0x20000), VP(0x30000), VP(0x40000), None) == BAD
    # what the calls refuse over such a pool comes before anything is launched
    att = lambda hq, **kw: lib.pa_attention(pool, 4, kw.get("q", DEV), pa.PA_BF16, hq, DEV, DEV, DEV, 4, kw.get("mb", 4), None, 0, 0.0,
                                            DEV, kw.get("ws"), kw.get("wsb", 0), None, None)
    assert att(5) == BAD and att(18) == NO and att(8, q=ODD) == BAD
    need = lib.pa_attention_workspace_bytes(pool, 4, 8, 400, None, 0)
    assert need > 0
    assert att(8, mb=400) == BAD
    assert att(8, mb=400, ws=VP(0x200000), wsb=need - 1) == BAD
    assert lib.pa_append_kv(pool, 4, ODD, DEV, pa.PA_BF16, DEV, DEV, DEV, 4, 4, None, None) == BAD
    assert lib.pa_append_kv(pool, 0, None, None, pa.PA_BF16, None, None, None, 4, 4, None, None) == OK


# ---------------------------------------------------------------------------- rotary positions --
@pytest.mark.parametrize("kw", [
    dict(rotary_dim=0), dict(rotary_dim=63), dict(rotary_dim=130), dict(rotary_dim=-2), dict(layout=2), dict(base=1.0),
    dict(base=-5.0), dict(base=float("nan")), dict(base=float("inf")), dict(scaling=5), dict(scaling=-1),
    dict(scaling=1, factor=0.0), dict(scaling=1, factor=-2.0), dict(scaling=1, factor=float("nan")),
    dict(scaling=2, factor=2.0, rotary_dim=2), dict(scaling=3, factor=2.0, low=1.0, high=32.0),
    dict(scaling=3, factor=2.0, low=0.0, high=32.0, original_positions=4096),
    dict(scaling=4, factor=2.0, low=4.0, high=4.0, original_positions=4096),
    dict(scaling=4, factor=2.0, low=1.0, high=float("inf"), original_positions=4096),
    dict(magnitude=-1.0), dict(magnitude=float("nan")),
    # frequencies that are no longer finite
    dict(scaling=1, factor=5e-324), dict(scaling=2, factor=1e-300, rotary_dim=4), dict(scaling=2, factor=1e300, rotary_dim=4)])
def test_rope_descriptions(lib, kw):
    st, h = create_rope(lib, **kw)
    assert st == BAD and not h.value


def test_rope_nulls(lib, rope):
    h = VP()
    assert lib.pa_rope_create(None, ctypes.byref(h)) == BAD
    assert lib.pa_rope_create(ctypes.byref(rope_desc()), None) == BAD
    assert lib.pa_rope_frequencies(None, None, None) == BAD
    assert lib.pa_rope_frequencies(rope, None, None) == OK
    lib.pa_rope_destroy(None)


def test_rope_rows_refusals(lib, rope):
    def call(r=rope, n=4, x=DEV, xs=512, out=VP(0x900000), os=512, dt=pa.PA_BF16, heads=8, d=64, pos=DEV):
        return lib.pa_rope_rows(r, n, x, xs, out, os, dt, heads, d, pos, 0, None)
    assert call(r=None) == BAD and call(n=-1) == BAD
    assert call(dt=pa.PA_FP8_E4M3) == BAD and call(dt=pa.PA_INT4) == BAD
    assert call(d=96) == NO and call(heads=0) == BAD and call(heads=1 << 17) == BAD
    assert call(x=None) == BAD and call(out=None) == BAD and call(pos=None) == BAD
    assert call(x=ODD) == BAD and call(out=ODD) == BAD
    assert call(xs=504) == BAD and call(xs=516) == BAD and call(os=511) == BAD and call(xs=-512) == BAD
    assert call(xs=514, dt=pa.PA_F32) == BAD
    assert call(out=DEV, xs=520) == BAD                      # in place with another stride
    assert call(n=0, x=None, out=None, pos=None) == OK
    st, wide = create_rope(lib, rotary_dim=128)
    assert st == OK
    assert call(r=wide) == BAD                               # rotary_dim beyond head_dim
    lib.pa_rope_destroy(wide)


def test_rope_append_refusals(lib, rope, pool):
    def call(p=pool, r=rope, n=4, q=DEV, qs=512, hq=8, qo=VP(0x900000), k=DEV, ks=128, v=DEV, vs=128, dt=pa.PA_BF16, ids=DEV, pos=DEV,
             bt=DEV, seqs=4, mb=4):
        return lib.pa_rope_append(p, r, n, q, qs, hq, qo, k, ks, v, vs, dt, ids, pos, bt, seqs, mb, None, None)
    assert call(p=None) == BAD and call(n=-1) == BAD and call(dt=pa.PA_FP8_E4M3) == BAD
    assert call(hq=-1) == BAD and call(seqs=0) == BAD and call(mb=0) == BAD
    for name in ("q", "qo", "k", "v", "ids", "pos", "bt"):
        assert call(**{name: None}) == BAD, name
    for name in ("q", "qo", "k", "v"):
        assert call(**{name: ODD}) == BAD, name
    assert call(qs=504) == BAD and call(ks=120) == BAD and call(vs=129) == BAD
    assert call(qo=DEV, qs=520) == BAD                       # in place, not contiguous
    assert call(n=0, q=None, qo=None, k=None, v=None, ids=None, pos=None, bt=None) == OK
    st, wide = create_rope(lib, rotary_dim=128)
    assert call(r=wide) == BAD
    lib.pa_rope_destroy(wide)


def test_read_refusals(lib, pool):
    def call(p=pool, n=4, ids=DEV, pos=DEV, bt=DEV, seqs=4, mb=4, k=DEV, v=DEV, dt=pa.PA_BF16):
        return lib.pa_read_kv(p, n, ids, pos, bt, seqs, mb, k, v, dt, None, None)
    assert call(p=None) == BAD and call(n=-1) == BAD and call(dt=pa.PA_INT4) == BAD
    assert call(seqs=0) == BAD and call(mb=-1) == BAD
    assert call(ids=None) == BAD and call(pos=None) == BAD and call(bt=None) == BAD
    assert call(k=ODD) == BAD and call(v=ODD) == BAD
    assert call(n=0, ids=None, pos=None, bt=None) == OK and call(k=None, v=None) == OK


# ------------------------------------------------------------------------------ prompt attention --
def test_prompt_refusals(lib):
    need = lib.pa_prompt_workspace_bytes(64, 3, 8, 2, 64)
    assert need > 0

    def call(n=64, seqs=3, q=DEV, qs=512, k=DEV, ks=128, v=DEV, vs=128, dt=pa.PA_BF16, hq=8, hkv=2, d=64, starts=DEV, out=DEV, ws=DEV,
             wsb=need):
        return lib.pa_prompt_attention(n, seqs, q, qs, k, ks, v, vs, dt, hq, hkv, d, starts, 0.0, out, None, ws, wsb, None, None)
    assert call(n=-1) == BAD and call(seqs=-1) == BAD and call(hq=7) == BAD and call(hkv=0) == BAD and call(hq=0) == BAD
    assert call(d=96) == NO and call(dt=pa.PA_F32) == NO and call(dt=pa.PA_INT4) == BAD
    for name in ("q", "k", "v", "out", "starts", "ws"):
        assert call(**{name: None}) == BAD, name
    for name in ("q", "k", "v", "out"):
        assert call(**{name: ODD}) == BAD, name
    assert call(qs=504) == BAD and call(ks=132) == BAD and call(vs=64) == BAD and call(vs=1 << 40) == BAD
    assert call(wsb=need - 1) == BAD and call(ws=VP(0x100010)) == BAD
    assert call(n=0, q=None, k=None, v=None, out=None) == OK and call(seqs=0) == OK
    assert call(n=(1 << 31) - 1, hq=1 << 14, hkv=2, qs=1 << 20) == NO


def test_prompt_workspace(lib):
    f = lib.pa_prompt_workspace_bytes
    assert f(-1, 1, 8, 2, 64) == 0 and f(64, -1, 8, 2, 64) == 0 and f(64, 1, 7, 2, 64) == 0 and f(64, 1, 8, 2, 80) == 0
    # one entry of 16 bytes for each tile of 128 (two heads) or 256 positions: at most one partial tile a sequence
    assert f(1 << 20, 1, 8, 2, 64) >= 256 + (1 << 13) * 16
    assert f(1000, 1000, 8, 2, 128) >= 256 + 1000 * 16
    assert f(1 << 20, 1, 3, 1, 64) >= 256 + (1 << 12) * 16


# -------------------------------------------------------------------------------------- tables --
def test_tables_refusals(lib):
    def grow(n=4, ids=DEV, lengths=DEV, new=DEV, free=DEV, count=DEV, left=DEV, pages=16, P=32, bt=DEV, seqs=4, mb=4, rs=DEV, ps=DEV, rows=8,
             rq=DEV, rp=DEV):
        return lib.pa_tables_grow(n, ids, lengths, new, free, count, left, pages, P, bt, seqs, mb, rs, ps, rows, rq, rp, None, None, None)

    def release(n=4, ids=DEV, lengths=DEV, free=DEV, count=DEV, pages=16, P=32, bt=DEV, seqs=4, mb=4):
        return lib.pa_tables_release(n, ids, lengths, None, free, count, pages, P, bt, seqs, mb, None, None)
    for call in (grow, release):
        assert call(n=-1) == BAD and call(pages=0) == BAD and call(seqs=0) == BAD and call(mb=0) == BAD
        assert call(P=48) == NO and call(P=8) == NO and call(P=512) == NO
        assert call(seqs=(1 << 19) + 1) == NO and call(mb=1 << 27, P=16) == NO
        for name in ("ids", "lengths", "free", "count", "bt"):
            assert call(**{name: None}) == BAD, name
    for name in ("new", "left", "rs", "ps", "rq", "rp"):
        assert grow(**{name: None}) == BAD, name
    assert grow(rows=-1) == BAD
    assert release(n=0, ids=None, lengths=None, free=None, count=None, bt=None) == OK


# --------------------------------------------------------------------------------- the binding --
def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


class FakePool:
    num_kv_heads, head_dim, k_pool = 2, 64, torch.zeros(16)
    handle = None


def test_binding_checks_types_and_shapes(lib):
    rope = pa.Rope(64)
    x, pos, bt = bf16(4, 8, 64), i32(4), i32(4, 4)
    with pytest.raises(TypeError, match="positions"):
        pa.rope_rows(rope, x, pos.long())
    with pytest.raises(ValueError, match="positions"):
        pa.rope_rows(rope, x, i32(5))
    with pytest.raises(ValueError, match="out"):
        pa.rope_rows(rope, x, pos, out=bf16(4, 8, 128))
    with pytest.raises(ValueError, match="heads"):
        pa.rope_rows(rope, bf16(4, 16, 64)[:, ::2], pos)
    with pytest.raises(ValueError, match="CUDA"):
        pa.rope_rows(rope, x, pos)
    kv = bf16(4, 2, 64)
    with pytest.raises(ValueError, match="k_new"):
        pa.rope_append(FakePool(), rope, x, bf16(4, 4, 64), bf16(4, 4, 64), pos, pos, bt, x)
    with pytest.raises(ValueError, match="q_out"):
        pa.rope_append(FakePool(), rope, x, kv, kv, pos, pos, bt, None)
    with pytest.raises(ValueError, match="dtype"):
        pa.rope_append(FakePool(), rope, x, kv, kv.float(), pos, pos, bt, x)
    with pytest.raises(TypeError, match="block_tables"):
        pa.rope_append(FakePool(), rope, x, kv, kv, pos, pos, bt.long(), x)
    with pytest.raises(ValueError, match="k_out"):
        pa.read_kv(FakePool(), pos, pos, bt)
    with pytest.raises(ValueError, match="v_out"):
        pa.read_kv(FakePool(), pos, pos, bt, v_out=bf16(4, 2, 128))
    with pytest.raises(ValueError, match="CUDA"):
        pa.read_kv(FakePool(), pos, pos, bt, k_out=kv)
    with pytest.raises(ValueError):
        pa.prompt_attention(x, kv, bf16(4, 2, 128), i32(3), x)
    with pytest.raises(ValueError, match="dtype"):
        pa.prompt_attention(x, kv.float(), kv.float(), i32(3), x)
    with pytest.raises(TypeError, match="row_starts"):
        pa.prompt_attention(x, kv, kv, i32(3).long(), x)
    with pytest.raises(ValueError, match="row_starts"):
        pa.prompt_attention(x, kv, kv, i32(0), x)
    with pytest.raises(ValueError, match="lse"):
        pa.prompt_attention(x, kv, kv, i32(3), x, lse=torch.zeros(4, 2))
    with pytest.raises(ValueError, match="CUDA"):
        pa.prompt_attention(x, kv, kv, i32(3), x)


@pytest.mark.parametrize("name,bad", [
    ("lengths", i32(3)), ("new_tokens", i32(5)), ("free_count", i32(2)), ("free_left", i32(2)), ("row_starts", i32(4)),
    ("page_starts", i32(6)), ("row_positions", i32(7)), ("block_tables", i32(4))])
def test_binding_checks_tables(lib, name, bad):
    a = dict(seq_ids=i32(4), lengths=i32(4), new_tokens=i32(4), free_pages=i32(16), free_count=i32(1), free_left=i32(1), page_size=16,
             block_tables=i32(4, 4), row_starts=i32(5), page_starts=i32(5), row_seqs=i32(8), row_positions=i32(8))
    with pytest.raises(ValueError, match="CUDA"):
        pa.tables_grow(**a)
    with pytest.raises(ValueError, match=name):
        pa.tables_grow(**dict(a, **{name: bad}))
    with pytest.raises(TypeError, match=name):
        pa.tables_grow(**dict(a, **{name: a[name].long()}))


def test_rope_frequencies_of_the_scalings(lib):
    """f_i of each scaling, from its formula in binary64: the two sides' powers, logarithms and a few operations differ by a
    few units of 2^-52 each, times the exponents' size (below 20): 1e-13 relative."""
    r, base, factor, old = 64, 10000.0, 8.0, 4096
    i = np.arange(r // 2)
    f = base ** (-2.0 * i / r)
    turns = old * f / (2 * np.pi)
    at = lambda t: r * np.log(old / (2 * np.pi * t)) / (2 * np.log(base))
    lo, hi = max(np.floor(at(32.0)), 0), min(np.ceil(at(1.0)), r - 1)
    ramp = np.clip((i - lo) / (hi - lo), 0, 1)
    bands = np.clip((turns - 1.0) / (4.0 - 1.0), 0, 1)
    want = {None: f, "linear": f / factor, "base": (base * factor ** (r / (r - 2))) ** (-2.0 * i / r),
            "ramp": f / factor * ramp + f * (1 - ramp), "bands": f / factor * (1 - bands) + f * bands}
    for name, w in want.items():
        got, m = pa.Rope(r, base=base, scaling=name, factor=factor, original_positions=old).frequencies()
        assert np.abs(got / w - 1).max() < 1e-13, name
        assert m == (pytest.approx(0.1 * np.log(factor) + 1) if name == "ramp" else 1.0)
