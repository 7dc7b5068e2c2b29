"""The cache operators without a GPU: refusals of the C ABI (nothing is
launched), the binding's checks, and pa_pages_trim."""
import ctypes
import types

import numpy as np
import pytest
import torch

import paged_kv_continuous_pa_gb300 as pa
from paged_kv_continuous_pa_gb300 import build as pa_build

DEV = ctypes.c_void_p(0x100000)


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return pa.load()


@pytest.fixture()
def pool(lib):
    d = pa.PoolDesc(num_pages=16, page_size=32, num_kv_heads=2, head_dim=64, kv_dtype=pa.PA_BF16, k_scale=1.0, v_scale=1.0)
    h = ctypes.c_void_p()
    assert lib.pa_pool_create(ctypes.byref(d), ctypes.c_void_p(0x10000), ctypes.c_void_p(0x20000), ctypes.byref(h)) == pa.PA_OK
    yield h
    lib.pa_pool_destroy(h)


def test_mass_refusals(lib, pool):
    def call(**kw):
        return lib.pa_attention_mass(kw.get("pool", pool), kw.get("n", 4), kw.get("q", DEV), kw.get("qd", pa.PA_BF16),
                                     kw.get("hq", 8), kw.get("seq", DEV), DEV, DEV, kw.get("seqs", 4), kw.get("mb", 4),
                                     kw.get("chunks"), kw.get("nc", 0), 0.0, kw.get("mass", DEV), kw.get("ws"),
                                     kw.get("wsb", 0), None, None)
    bad, unsupported = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED
    assert call(pool=None) == bad
    assert call(n=-1) == bad
    assert call(n=0, q=None, mass=None) == pa.PA_OK
    assert call(q=None) == bad and call(seq=None) == bad and call(mass=None) == bad
    assert call(q=ctypes.c_void_p(0x100008)) == bad and call(mass=ctypes.c_void_p(0x100004)) == bad
    assert call(hq=5) == bad and call(hq=0) == bad and call(hq=18) == unsupported
    assert call(qd=pa.PA_FP8_E4M3) == bad
    assert call(seqs=0) == bad and call(mb=0) == bad
    assert call(mb=1 << 27) == unsupported
    two = (pa.Chunk * 2)(pa.Chunk(0, 3), pa.Chunk(2, 2))
    assert call(chunks=two, nc=2) == bad
    assert call(chunks=None, nc=1) == bad
    # a window on the tile path needs its workspace
    win = (pa.Chunk * 1)(pa.Chunk(0, 64))
    need = lib.pa_attention_mass_workspace_bytes(pool, 64, 8, 4, win, 1)
    if need:
        assert call(n=64, chunks=win, nc=1) == bad
        assert call(n=64, chunks=win, nc=1, ws=DEV, wsb=need - 1) == bad
        assert call(n=64, chunks=win, nc=1, ws=ctypes.c_void_p(0x100010), wsb=need) == bad
    assert lib.pa_attention_mass_workspace_bytes(None, 64, 8, 4, win, 1) == 0
    assert lib.pa_attention_mass_workspace_bytes(pool, 64, 7, 4, win, 1) == 0


def test_select_refusals(lib):
    def call(**kw):
        return lib.pa_evict_select(kw.get("n", 2), kw.get("seq", DEV), kw.get("len", DEV), kw.get("mass", DEV),
                                   kw.get("seqs", 4), kw.get("heads", 2), kw.get("tokens", 100), kw.get("budget", 10),
                                   kw.get("first", 0), kw.get("last", 0), kw.get("keep", DEV), None, None, None)
    bad = pa.PA_ERR_INVALID_ARG
    assert call(n=-1) == bad
    assert call(n=0, seq=None) == pa.PA_OK
    for name in ("seq", "len", "mass", "keep"):
        assert call(**{name: None}) == bad
    for name in ("seqs", "heads", "tokens", "budget"):
        assert call(**{name: 0}) == bad
    assert call(first=-1) == bad and call(last=-1) == bad
    assert call(first=6, last=5) == bad and "budget" in pa.last_error()
    assert call(first=0x7fffffff, last=0x7fffffff) == bad
    assert call(n=0x7fffffff) == pa.PA_ERR_UNSUPPORTED and call(tokens=(1 << 30) + 1) == pa.PA_ERR_UNSUPPORTED


def test_compact_refusals(lib, pool):
    def call(**kw):
        return lib.pa_evict_compact(kw.get("pool", pool), kw.get("n", 2), kw.get("seq", DEV), None, kw.get("len", DEV),
                                    kw.get("keep", DEV), kw.get("budget", 10), kw.get("bt", DEV), kw.get("seqs", 4),
                                    kw.get("mb", 4), None, None, None)
    bad = pa.PA_ERR_INVALID_ARG
    assert call(pool=None) == bad and call(n=-1) == bad
    assert call(n=0, seq=None) == pa.PA_OK
    for name in ("seq", "len", "keep", "bt"):
        assert call(**{name: None}) == bad
    for name in ("seqs", "mb", "budget"):
        assert call(**{name: 0}) == bad
    assert call(mb=1 << 27) == pa.PA_ERR_UNSUPPORTED


def test_beam_select_refusals(lib):
    def call(**kw):
        return lib.pa_beam_select(kw.get("n", 2), kw.get("b", 4), kw.get("v", 100), kw.get("logits", DEV),
                                  kw.get("dt", pa.PA_F32), kw.get("stride", 100), kw.get("scores", DEV), None, 0,
                                  kw.get("out", 8), kw.get("parents", DEV), DEV, DEV, kw.get("ws", DEV),
                                  kw.get("wsb", 1 << 20), None)
    bad, unsupported = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED
    assert call(n=-1) == bad
    assert call(n=0, logits=None, ws=None) == pa.PA_OK
    for name in ("logits", "scores", "parents", "ws"):
        assert call(**{name: None}) == bad
    assert call(b=0) == bad and call(v=0) == bad and call(out=0) == bad
    assert call(b=33) == unsupported and call(out=65) == unsupported and call(v=(1 << 20) + 1, stride=1 << 21) == unsupported
    assert call(dt=pa.PA_FP8_E4M3) == bad
    assert call(stride=99) == bad
    assert call(logits=ctypes.c_void_p(0x100002)) == bad
    need = lib.pa_beam_workspace_bytes(2, 4, 100, 8)
    assert need > 0 and need % 256 == 0
    assert call(wsb=need - 1) == bad and call(ws=ctypes.c_void_p(0x100010)) == bad
    for args in ((0, 4, 100, 8), (2, 33, 100, 8), (2, 4, 0, 8), (2, 4, 100, 65), (2, 4, 100, 0)):
        assert lib.pa_beam_workspace_bytes(*args) == 0


def test_reorder_refusals(lib, pool):
    def call(**kw):
        return lib.pa_beam_reorder(kw.get("pool", pool), kw.get("n", 2), kw.get("b", 4), kw.get("seq", DEV),
                                   kw.get("parents", DEV), kw.get("len", DEV), kw.get("bt", DEV), kw.get("seqs", 8),
                                   kw.get("mb", 4), kw.get("state"), kw.get("bytes", 0), None, None)
    bad, unsupported = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED
    assert call(pool=None) == bad and call(n=-1) == bad and call(b=0) == bad
    assert call(n=0, seq=None) == pa.PA_OK
    assert call(b=33) == unsupported and call(n=65536) == unsupported and call(mb=1 << 27) == unsupported
    for name in ("seq", "parents", "len", "bt"):
        assert call(**{name: None}) == bad
    assert call(state=DEV, bytes=0) == bad and call(state=DEV, bytes=6) == bad
    assert call(state=ctypes.c_void_p(0x100002), bytes=8) == bad


# ------------------------------------------------------------- the binding --

POOL = types.SimpleNamespace(head_dim=64, num_kv_heads=2, page_size=16, handle=None, k_pool=torch.zeros(1))


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def test_mass_binding():
    good = dict(q=torch.zeros(3, 4, 64), seq_ids=i32(3), positions=i32(3), block_tables=i32(2, 5), mass=torch.zeros(2, 2, 80))

    def call(**kw):
        return pa.attention_mass(POOL, **{**good, **kw})
    with pytest.raises(ValueError, match="CUDA"):
        call()
    with pytest.raises(TypeError, match="mass"):
        call(mass=torch.zeros(2, 2, 80, dtype=torch.float64))
    with pytest.raises(ValueError, match="mass"):
        call(mass=torch.zeros(2, 2, 79))
    with pytest.raises(TypeError, match="positions"):
        call(positions=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="q has shape"):
        call(q=torch.zeros(3, 4, 128))


def test_evict_binding():
    good = dict(mass=torch.zeros(2, 2, 80), seq_ids=i32(3), lengths=i32(3), keep=i32(3, 2, 8))

    def call(**kw):
        return pa.evict_select(**{**good, **kw})
    with pytest.raises(ValueError, match="CUDA"):
        call()
    with pytest.raises(ValueError, match="keep"):
        call(keep=i32(3, 1, 8))
    with pytest.raises(TypeError, match="keep"):
        call(keep=torch.zeros(3, 2, 8, dtype=torch.int64))
    with pytest.raises(TypeError, match="mass"):
        call(mass=torch.zeros(2, 2, 80, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="kept_lengths"):
        call(kept_lengths=good["lengths"])
    with pytest.raises(ValueError, match="lengths"):
        call(lengths=i32(2))
    more = dict(keep=i32(3, 2, 8), seq_ids=i32(3), lengths=i32(3), block_tables=i32(4, 5))

    def compact(**kw):
        return pa.evict_compact(POOL, **{**more, **kw})
    with pytest.raises(ValueError, match="CUDA"):
        compact()
    with pytest.raises(ValueError, match="mass"):
        compact(mass=torch.zeros(4, 2, 81))
    with pytest.raises(ValueError, match="dst_seq_ids"):
        compact(dst_seq_ids=i32(4))
    with pytest.raises(ValueError, match="keep"):
        compact(keep=i32(3, 16))


def test_beam_binding():
    good = dict(logits=torch.zeros(2, 4, 100), scores=torch.zeros(2, 4), parents=i32(2, 8), tokens=i32(2, 8),
                out_scores=torch.zeros(2, 8))

    def call(**kw):
        return pa.beam_select(**{**good, **kw})
    with pytest.raises(ValueError, match="CUDA"):
        call()
    with pytest.raises(ValueError, match="CUDA"):
        call(logits=torch.zeros(2, 4, 104)[:, :, :100])
    with pytest.raises(ValueError, match="rows"):
        call(logits=torch.zeros(2, 100, 4).transpose(1, 2))
    with pytest.raises(ValueError, match="rows"):
        call(logits=torch.zeros(2, 8, 100)[:, :4])
    with pytest.raises(ValueError, match="scores"):
        call(scores=torch.zeros(2, 5))
    with pytest.raises(TypeError, match="tokens"):
        call(tokens=torch.zeros(2, 8, dtype=torch.int64))
    with pytest.raises(TypeError, match="finished"):
        call(finished=torch.zeros(2, 4, dtype=torch.bool))
    more = dict(parents=i32(2, 4), seq_ids=i32(2, 4), lengths=i32(2), block_tables=i32(8, 5))

    def reorder(**kw):
        return pa.beam_reorder(POOL, **{**more, **kw})
    with pytest.raises(ValueError, match="CUDA"):
        reorder()
    with pytest.raises(ValueError, match="seq_ids"):
        reorder(seq_ids=i32(8))
    with pytest.raises(ValueError, match="state"):
        reorder(state=torch.zeros(7, 3))


# ------------------------------------------------------------------- trim --

def test_trim_gives_pages_back(lib):
    p = pa.Pages(20, 16, 3, 10)
    assert p.admit(0, 100, 20)[0] == pa.PA_OK  # 8 pages
    assert p.admit(1, 40, 0)[0] == pa.PA_OK    # 3 pages
    row = p.block_tables[0].copy()
    p.trim(0, 33)                              # 3 pages stay
    assert p.free_count() == 20 - 3 - 3
    assert np.array_equal(p.block_tables[0], np.concatenate([row[:3], [-1] * 7]))
    p.trim(0, 500)                             # nothing more to give
    assert p.free_count() == 14
    assert p.admit(2, 160, 0)[0] == pa.PA_OK   # the freed pages serve again
    p.trim(0, 0)
    assert (p.block_tables[0] == -1).all()
    p.release(0)
    p.release(1)
    p.release(2)
    assert p.free_count() == 20


def test_trim_respects_shared_pages(lib):
    p = pa.Pages(20, 16, 3, 10)
    assert p.admit(0, 64, 0)[0] == pa.PA_OK
    assert p.admit(1, 64, 16, 0, 64)[0] == pa.PA_OK
    shared = p.block_tables[0][3]
    assert p.refcount(shared) == 2
    p.trim(0, 16)
    assert p.refcount(shared) == 1 and p.free_count() == 20 - 5
    assert p.block_tables[1][3] == shared
    p.release(1)
    assert p.refcount(shared) == 0


def test_trim_refusals(lib):
    p = pa.Pages(8, 16, 2, 4)
    for seq, tokens in ((0, 5), (-1, 5), (2, 5)):
        with pytest.raises(pa.PaError):
            p.trim(seq, tokens)
    assert p.admit(0, 30, 0)[0] == pa.PA_OK
    with pytest.raises(pa.PaError):
        p.trim(0, -1)
    assert lib.pa_pages_trim(None, 0, 0, None) == pa.PA_ERR_INVALID_ARG
    assert lib.pa_pages_trim(p.handle, 0, 16, None) == pa.PA_OK and p.free_count() == 7


def test_longest_block_table(lib, pool):
    """Tables of more than 2^30 tokens are refused (positions and steps beyond them stay 32-bit)."""
    longest = (1 << 30) // 32

    def mass(blocks):
        return lib.pa_attention_mass(pool, 4, None, pa.PA_BF16, 8, None, None, None, 4, blocks, None, 0, 0.0, None, None,
                                     0, None, None)

    def compact(blocks):
        return lib.pa_evict_compact(pool, 0, None, None, None, None, 8, None, 4, blocks, None, None, None)

    assert mass(longest) == pa.PA_ERR_INVALID_ARG and "NULL" in pa.last_error()  # as far as its pointers
    assert mass(longest + 1) == pa.PA_ERR_UNSUPPORTED
    assert compact(longest) == pa.PA_OK
    assert compact(longest + 1) == pa.PA_ERR_UNSUPPORTED


def test_numbers_beyond_32_bits(lib):
    """They are refused, not cut to their lower bits."""
    mass, three = torch.zeros(2, 2, 80), i32(3)
    for name in ("keep_first", "keep_last"):
        for value in (1 << 32, (1 << 32) + 4, -(1 << 32)):
            with pytest.raises(ValueError, match=name):
                pa.evict_select(mass, three, i32(3), i32(3, 2, 8), **{name: value})
    with pytest.raises(ValueError, match="end_token"):
        pa.beam_select(torch.zeros(2, 4, 100), torch.zeros(2, 4), i32(2, 8), i32(2, 8), torch.zeros(2, 8), end_token=1 << 32)
    p = pa.Pages(20, 16, 3, 10)
    assert p.admit(0, 100, 20)[0] == pa.PA_OK
    for args in ((0, 1 << 32), ((1 << 32), 0)):
        with pytest.raises(ValueError, match="32 bits"):
            p.trim(*args)
    assert p.free_count() == 12


def test_select_does_not_write_its_inputs(lib):
    """The C entry refuses counts that would go over what other CTAs of the call still read."""
    other = [ctypes.c_void_p(0x200000 + 0x1000 * i) for i in range(4)]

    def call(kept):
        return lib.pa_evict_select(2, other[0], other[1], other[2], 4, 2, 100, 10, 0, 0, other[3], kept, None, None)
    assert call(other[0]) == pa.PA_ERR_INVALID_ARG and "kept_lengths" in pa.last_error()
    assert call(other[1]) == pa.PA_ERR_INVALID_ARG and "kept_lengths" in pa.last_error()
