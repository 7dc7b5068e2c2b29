"""README's eviction example, run as it stands: the sequence goes on to the end
of its answer, and the pages that it gave back belong to another one."""
import os
import re
import types

import numpy as np
import pytest
import torch

import paged_kv_continuous_pa_gb300 as pa
from paged_kv_continuous_pa_gb300 import build as pa_build

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")
P, BLOCKS, BUDGET, TO_COME = 16, 30, 96, 20  # the budget ends with a page: the next token needs the one behind it
LENGTHS = [400, 90, 250]


def example():
    with open(README) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    return next(b for b in blocks if "evict_compact" in b)


def admitted():
    pages = pa.Pages(100, P, 4, BLOCKS)
    for slot, n in enumerate(LENGTHS):
        assert pages.admit(slot, n, TO_COME)[0] == pa.PA_OK
    return pages


def i32(x, device):
    return torch.tensor(x, dtype=torch.int32, device=device)


def names(pages, device, **more):
    n, slots = len(LENGTHS), range(len(LENGTHS))
    return dict(torch=torch, pages=pages, num_seqs=4, max_blocks=BLOCKS, P=P, Hkv=2, Hq=4, n_rows=n, n=n, chunks=[],
                budget=BUDGET, to_come=TO_COME, slots=i32(list(slots), device), lengths=i32(LENGTHS, device),
                kept_lengths=torch.empty(n, dtype=torch.int32, device=device), seq_ids=i32(list(slots), device),
                positions=i32([x - 1 for x in LENGTHS], device),
                block_tables=torch.from_numpy(pages.block_tables.copy()).to(device), **more)


def test_tokens_to_come_keep_their_pages():
    pa_build.build()
    pages = admitted()
    calls = types.SimpleNamespace(mass_workspace_bytes=lambda *a: 0, attention_mass=lambda *a, **kw: None,
                                  evict_select=lambda *a, **kw: None, evict_compact=lambda *a, **kw: None)
    env = names(pages, "cpu", pa=calls, pool=None, q=None)
    held = pages.block_tables.copy()
    for slot, length in enumerate(LENGTHS):
        exec(example().replace('device="cuda"', 'device="cpu"'), {**env, "slot": slot, "length": length})
    assert pages.free_count() == 100 - sum(-(-(min(x, BUDGET) + TO_COME) // P) for x in LENGTHS)
    assert pages.admit(3, BLOCKS * P, 0)[0] == pa.PA_OK
    others = set(pages.block_tables[3].tolist())
    table = env["block_tables"].numpy()
    for slot, length in enumerate(LENGTHS):
        kept = min(length, BUDGET)
        for t in range(kept + TO_COME):
            assert table[slot, t // P] == held[slot, t // P] >= 0
        assert not others & set(table[slot].tolist())
    assert np.array_equal(table[:3], pages.block_tables[:3])


@pytest.mark.gpu
def test_the_sequence_goes_on():
    """Every token still to come is appended beside a new owner of the freed pages, and attention sees both."""
    Hkv, G, D = 2, 2, 64
    g = torch.Generator("cuda").manual_seed(5)
    pages = admitted()
    k_pool, v_pool = (torch.zeros(100, Hkv, P, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pool = pa.Pool(k_pool, v_pool)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def rows(n, heads):
        return torch.randn(n, heads, D, device="cuda", generator=g).bfloat16()

    env = names(pages, "cuda", pa=pa, pool=pool, q=rows(len(LENGTHS), Hkv * G))
    tables = env["block_tables"]

    def append(slot, first, k, v):
        n = k.shape[0]
        pa.append_kv(pool, k, v, i32([slot] * n, "cuda"), i32(list(range(first, first + n)), "cuda"), tables, status=status)

    cache = {}
    for slot, n in enumerate(LENGTHS):
        cache[slot] = rows(n, Hkv), rows(n, Hkv)
        append(slot, 0, *cache[slot])
    env.update(slots=i32([0], "cuda"), lengths=i32(LENGTHS[:1], "cuda"), n=1, kept_lengths=i32([0], "cuda"),
               slot=0, length=LENGTHS[0])
    # (keep_last of the example and its first tokens fit in the budget)
    exec(example(), env)
    keep = env["keep"][0].long()
    assert env["kept_lengths"].tolist() == [BUDGET]
    hist = [torch.stack([x[keep[h], h] for h in range(Hkv)], dim=1) for x in cache[0]]
    assert pages.admit(3, BLOCKS * P, 0)[0] == pa.PA_OK
    tables[3].copy_(torch.from_numpy(pages.block_tables[3]))
    cache[3] = rows(BLOCKS * P, Hkv), rows(BLOCKS * P, Hkv)
    append(3, 0, *cache[3])
    for t in range(BUDGET, BUDGET + TO_COME):
        new = rows(1, Hkv), rows(1, Hkv)
        append(0, t, *new)
        hist = [torch.cat([x, y]) for x, y in zip(hist, new)]
        q = rows(2, Hkv * G)
        out = torch.empty_like(q)
        pa.attention(pool, q, i32([0, 3], "cuda"), i32([t, BLOCKS * P - 1], "cuda"), tables, out, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        for i, (kk, vv) in enumerate((hist, cache[3])):
            kk, vv = (x.double().transpose(0, 1) for x in (kk, vv))
            s = torch.einsum("hgd,htd->hgt", q[i].double().view(Hkv, G, D), kk) / D ** 0.5
            ref = torch.einsum("hgt,htd->hgd", torch.softmax(s, dim=2), vv).reshape(Hkv * G, D)
            err = (out[i].double() - ref).abs()
            assert ((err <= 2e-3) | (err <= 1e-2 * ref.abs())).all()
