"""Random paged caches on the GPU, and 64-bit references of the cache
operators written from their definitions (torch, float64)."""
from __future__ import annotations

import math
from types import SimpleNamespace

import torch

import paged_kv_continuous_pa_gb300 as pa

KV = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.uint8}


def random_rows(shape, kv, g):
    """N(0, 1) cache elements in the pool's storage type (fp8: codes of N(0, 1) * 32)."""
    x = torch.randn(shape, generator=g)
    if kv == "e4m3":
        return (x * 32).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.to(KV[kv])


def values(x, scale=1.0):
    """Stored elements as float64 (scale: fp8 scale, a float or [Hkv, 1, 1])."""
    if x.dtype == torch.uint8:
        return x.view(torch.float8_e4m3fn).to(torch.float64) * scale
    return x.to(torch.float64)


def bits(x):
    return x.contiguous().reshape(-1).view(torch.uint8)


def make_cache(lengths, Hkv=2, D=64, P=16, kv="bf16", seed=0, spare_blocks=1, slots=None, device="cuda"):
    """A pool whose sequences hold `lengths` tokens; every other slot is NaN.
    Pages are in random order, sequence i sits in slot slots[i]."""
    g = torch.Generator().manual_seed(seed)
    n = len(lengths)
    num_seqs = n + 2 if slots is None else max(max(slots) + 1, n)
    slots = torch.randperm(num_seqs, generator=g)[:n].tolist() if slots is None else list(slots)
    max_blocks = max(1, max(-(-x // P) for x in lengths) + spare_blocks)
    num_pages = num_seqs * max_blocks
    order = torch.randperm(num_pages, generator=g).view(num_seqs, max_blocks).to(torch.int32)
    shape = (num_pages, Hkv, P, D)
    pools = []
    for _ in range(2):
        pool = torch.full(shape, 0x7F, dtype=torch.uint8) if kv == "e4m3" else torch.full(shape, float("nan"), dtype=KV[kv])
        for i, length in enumerate(lengths):
            rows = random_rows((length, Hkv, D), kv, g)
            t = torch.arange(length)
            pool[order[slots[i]][t // P].long(), :, t % P] = rows
        pools.append(pool.to(device))
    scale = 1.0
    if kv == "e4m3":
        scale = (torch.rand(Hkv, generator=g) * 0.02 + 0.02).to(torch.float32)
    k, v = pools
    handle = pa.Pool(k, v, scale.numpy(), scale.numpy()) if kv == "e4m3" else pa.Pool(k, v)
    wide = scale.to(torch.float64).view(-1, 1, 1).to(device) if kv == "e4m3" else 1.0
    return SimpleNamespace(pool=handle, k=k, v=v, kv=kv, tables=order.to(device), slots=slots, lengths=list(lengths),
                           Hkv=Hkv, D=D, P=P, num_seqs=num_seqs, max_blocks=max_blocks, scale=wide,
                           max_tokens=max_blocks * P)


def cached(c, pool, slot, length, tables=None):
    """[Hkv, length, D] stored elements of a slot's first tokens."""
    tables = c.tables if tables is None else tables
    t = torch.arange(length, device=pool.device)
    return pool[tables[slot][t // c.P].long(), :, t % c.P].transpose(0, 1)


def mass_of_rows(c, q, seq_ids, positions, softmax_scale=None):
    """float64 [num_seqs, Hkv, max_tokens] added weights of the given rows, and
    the largest sum of |q_d k_d| * scale over them (for error bounds)."""
    sm = softmax_scale or 1.0 / math.sqrt(c.D)
    out = torch.zeros(c.num_seqs, c.Hkv, c.max_tokens, dtype=torch.float64, device=q.device)
    G = q.shape[1] // c.Hkv
    big = 0.0
    for r, (s, p) in enumerate(zip(seq_ids, positions)):
        k = values(cached(c, c.k, s, p + 1), c.scale)
        qr = q[r].to(torch.float64).view(c.Hkv, G, c.D)
        w = torch.softmax(torch.einsum("hgd,htd->hgt", qr, k) * sm, dim=2)
        big = max(big, float(torch.einsum("hgd,htd->hgt", qr.abs(), k.abs()).max()) * sm)
        out[s, :, :p + 1] += w.sum(dim=1)
    return out, big


def mass_bound(c, added, before, big, rows, G):
    """Elementwise error bound of the FP32 kernel.

    A score (log2 units) is a dot product of D terms on a scaled query: its
    error is at most (D + 8) roundings of 2^-23 (twice the FP32 half step, as
    tensor cores may truncate) of the sum of the terms' sizes, `big` * log2(e);
    it enters a weight through the exponential and through the log-sum-exp
    (factor 2 ln 2).  The weight sum has at most max_tokens additions and the
    accumulation over rows and heads rows * G + 2, each a half step 2^-24;
    ex2.approx adds 2^-22 twice.  Adding to the buffer rounds once more.
    Weights below 2^-126 are flushed."""
    rel = 2 * math.log(2) * (c.D + 8) * 2.0 ** -23 * big * math.log2(math.e)
    rel += (c.max_tokens + rows * G + 2) * 2.0 ** -24 + 2.0 ** -21
    return rel * added + 2.0 ** -23 * (added + before) + rows * G * 2.0 ** -126


def select_ref(mass, length, budget, first, last):
    """Kept tokens of one (sequence, kv head), ascending (python, exact)."""
    if length <= budget:
        return list(range(length))
    w = [(-math.inf, 1) if x != x else (x, 0) for x in mass[:length].tolist()]
    middle = range(first, length - last)
    best = sorted(middle, key=lambda t: (w[t][1], -w[t][0], t))[:budget - first - last]
    return sorted(list(range(first)) + best + list(range(length - last, length)))
