"""The operators of a serving step around the paged cache, as cases to be measured.

  tables   block tables, the row list of a step and its slot map, made on the
           GPU from the requests' lengths and a stack of free pages
  rope     rotary positions: a step's queries rotated, its keys rotated and
           stored in their page slots, its values stored
  prompt   causal attention over whole prompts packed one behind the other
  append4  a step's keys and values stored in a 4-bit pool, and read back
  attend4  single-token attention over a 4-bit pool

With ``own`` false, run() computes them in elementary torch operations; with
``own`` true it makes the library's calls.  Sizes are those of this
repository's workloads (batched decode: 512 sequences of 64..2662 tokens, 16
query and 8 kv heads of 128; long context: 32768 tokens, 32 query heads; pages
of 16 to 256 tokens) or generic ones.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.uint8}
SIZE = {"f32": 4, "bf16": 2, "e4m3": 1}
SCALE = 1.0 / 32.0  # of the fp8 pools


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # eight conversations, one token each: the smallest call
        {"name": "tables 8 decode", "op": "tables", "seqs": 8, "lo": 100, "hi": 2662, "new_lo": 1, "new_hi": 1,
         "page": 32, "blocks": 128},
        # a batch of prompts enters an empty cache
        {"name": "tables 512 prompts", "op": "tables", "seqs": 512, "lo": 0, "hi": 0, "new_lo": 64, "new_hi": 2662,
         "page": 16, "blocks": 256},
        # a decode step's projections, one packed qkv row per sequence
        {"name": "rope 64 decode", "op": "rope", "seqs": 64, "lo": 1, "hi": 1, "start": 2600, "hq": 16, "hkv": 8,
         "d": 128, "rot": 128, "layout": "half", "scaling": "none", "page": 32, "kv": "bf16", "x": "bf16",
         "packed": True},
        # prompts of 32768 tokens in all, positions stretched for a long context, half of each head rotated
        {"name": "rope 32768 far", "op": "rope", "seqs": 8, "lo": 4096, "hi": 4096, "start": 28000, "hq": 32, "hkv": 8,
         "d": 128, "rot": 64, "layout": "interleaved", "scaling": "ramp", "page": 64, "kv": "bf16", "x": "bf16",
         "packed": True},
        # one short prompt: the call's latency
        {"name": "prompt 1x77", "op": "prompt", "seqs": 1, "lo": 77, "hi": 77, "hq": 16, "hkv": 8, "d": 128, "pad": 0,
         "packed": False},
        # a batch of ragged prompts behind one packed projection
        {"name": "prompt 64 ragged", "op": "prompt", "seqs": 64, "lo": 64, "hi": 2662, "hq": 16, "hkv": 8, "d": 128,
         "pad": 37, "packed": True},
        # one long document
        {"name": "prompt 1x16384", "op": "prompt", "seqs": 1, "lo": 16384, "hi": 16384, "hq": 32, "hkv": 8, "d": 128,
         "pad": 0, "packed": True},
        # a decode step's new tokens
        {"name": "append4 64 rows", "op": "append4", "seqs": 64, "lo": 1, "hi": 1, "start": 900, "hkv": 8, "d": 128,
         "page": 32, "x": "bf16"},
        # long prompts enter the cache
        {"name": "append4 16384 rows", "op": "append4", "seqs": 16, "lo": 700, "hi": 1348, "start": 0, "hkv": 8,
         "d": 128, "page": 16, "x": "bf16"},
        # a few short conversations
        {"name": "attend4 4 short", "op": "attend4", "seqs": 4, "lo": 64, "hi": 900, "hq": 16, "hkv": 8, "d": 128,
         "page": 32, "x": "bf16"},
        # the batched decode step
        {"name": "attend4 512 ragged", "op": "attend4", "seqs": 512, "lo": 64, "hi": 2662, "hq": 16, "hkv": 8,
         "d": 128, "page": 32, "x": "bf16"},
        # long contexts, where a small cache pays most
        {"name": "attend4 64 long", "op": "attend4", "seqs": 64, "lo": 30000, "hi": 32768, "hq": 32, "hkv": 8,
         "d": 128, "page": 16, "x": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "rope", "rope", "prompt", "prompt", "append4", "attend4", "attend4"])
    page = rng.choice([16, 32, 64, 128, 256])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.randint(1, 8)
    x = rng.choice(["bf16", "bf16", "f32"])
    if op == "tables":
        prompts = rng.random() < 0.5
        seqs = _log(rng, 1, 2048)
        new = _log(rng, 1, max(1, min(8192, 700000 // seqs))) if prompts else 1
        hi = 0 if prompts and rng.random() < 0.5 else _log(rng, 1, 4096)
        return {"op": op, "seqs": seqs, "lo": hi // 3, "hi": hi, "new_lo": max(1, new // 4) if prompts else 0,
                "new_hi": new, "page": page, "blocks": -(-(hi + new) // page) + rng.randint(0, 3)}
    if op == "rope":
        seqs = _log(rng, 1, 256)
        most = 32768 * 40 * 128 // ((hq + 2 * hkv) * d * seqs)
        hi = rng.choice([1, _log(rng, 1, 8192)])
        hi = max(1, min(hi, most * (2 if x == "bf16" else 1) // 2))
        return {"op": op, "seqs": seqs, "lo": max(1, hi // 3), "hi": hi, "start": rng.choice([0, _log(rng, 1, 400000)]),
                "hq": hq, "hkv": hkv, "d": d, "rot": rng.choice([d, d, d // 2, d // 4]),
                "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "base", "ramp", "bands"]), "page": page,
                "kv": rng.choice(["bf16", "bf16", "f32", "e4m3"]), "x": x, "packed": rng.random() < 0.5}
    if op == "prompt":
        hi = _log(rng, 1, 16384)
        # neither more work than the longest prompt nor more room than its plain form takes
        most = 16384 * 16384 * 32 * 128 // (hi * hi * hq * 128)
        if most < 1:
            hi, most = 4096, max(1, 16 * 32 // hq)
        return {"op": op, "seqs": max(1, min(_log(rng, 1, 128), most)), "lo": max(1, hi // rng.choice([1, 4, 30])),
                "hi": hi, "hq": hq, "hkv": hkv, "d": d, "pad": rng.choice([0, 0, 19, 300]),
                "packed": rng.random() < 0.5}
    if op == "append4":
        seqs = _log(rng, 1, 256)
        hi = max(1, min(_log(rng, 1, 4096), 16384 * 8 * 128 // (seqs * hkv * d)))
        return {"op": op, "seqs": seqs, "lo": max(1, hi // 2), "hi": hi, "start": rng.choice([0, rng.randint(1, 3000)]),
                "hkv": hkv, "d": d, "page": page, "x": x}
    hi = _log(rng, 1, 32768)
    seqs = max(1, min(_log(rng, 1, 512), 64 * 32768 * 8 * 128 // (hi * hkv * d)))
    return {"op": op, "seqs": seqs, "lo": max(1, hi // rng.choice([1, 4, 30])), "hi": hi, "hq": hq, "hkv": hkv, "d": d,
            "page": page, "x": x}


# ----------------------------------------------------------------- inputs --

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _whole(n, lo, hi, g):
    return torch.randint(lo, hi + 1, (n,), device=DEV, generator=g, dtype=torch.int32)


def _spread(case, g):
    """Lengths spread evenly over lo..hi, the same ones in each seed's order: the rows in all go by the case alone."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    lengths = torch.linspace(lo, hi, n, dtype=torch.float64, device=DEV).round().to(torch.int32) if n > 1 else \
        torch.full((1,), hi, dtype=torch.int32, device=DEV)
    return lengths[torch.randperm(n, device=DEV, generator=g)]


def _normal(shape, dtype, g):
    return torch.empty(shape, device=DEV, dtype=dtype).normal_(generator=g)


def _library():
    import paged_kv_continuous_pa_gb300 as pa
    return pa


def prepare(case, seed):
    g = _generator(seed)
    return {"tables": _prepare_tables, "rope": _prepare_rope, "prompt": _prepare_prompt, "append4": _prepare_append4,
            "attend4": _prepare_attend4}[case["op"]](case, g)


def _prepare_tables(case, g):
    n, page, blocks = case["seqs"], case["page"], case["blocks"]
    lengths = _whole(n, case["lo"], case["hi"], g)
    new = _whole(n, case["new_lo"], case["new_hi"], g)
    slots = n + n // 4 + 1
    pages = slots * blocks
    order = torch.randperm(pages, device=DEV, generator=g).to(torch.int32)
    tables = order.view(slots, blocks).clone()
    seqs = torch.randperm(slots, device=DEV, generator=g)[:n].to(torch.int32)
    # pages held: those of the tokens cached so far; every other page is free
    held = torch.zeros(slots, dtype=torch.int64, device=DEV)
    held[seqs.long()] = (lengths.long() + page - 1) // page
    unused = torch.arange(blocks, device=DEV) >= held.view(-1, 1)
    free = tables[unused]
    free = free[torch.randperm(free.numel(), device=DEV, generator=g)]
    stack = torch.full((pages,), -1, dtype=torch.int32, device=DEV)
    stack[:free.numel()] = free
    tables[unused] = -1
    rows = n * case["new_hi"]
    st = {"case": case, "seqs": seqs, "lengths": lengths, "new": new, "free": stack, "tables": tables,
          "count": torch.tensor([free.numel()], dtype=torch.int32, device=DEV),
          "left": torch.zeros(1, dtype=torch.int32, device=DEV),
          "row_starts": torch.zeros(n + 1, dtype=torch.int32, device=DEV),
          "page_starts": torch.zeros(n + 1, dtype=torch.int32, device=DEV),
          "row_seqs": torch.full((rows,), -1, dtype=torch.int32, device=DEV),
          "row_positions": torch.full((rows,), -1, dtype=torch.int32, device=DEV),
          "row_slots": torch.full((rows,), -1, dtype=torch.int64, device=DEV)}
    if own:
        st["pa"] = _library()
    return st


def _rows(case, g):
    """Sequence ids and positions of a step in which every sequence has lo..hi new tokens, and tables with its pages."""
    n, page, start = case["seqs"], case["page"], case["start"]
    new = _spread(case, g)
    first = torch.randint(start // 2, start + 1, (n,), device=DEV, generator=g)
    slots = torch.randperm(n, device=DEV, generator=g)
    total = int(new.sum())
    seq = torch.repeat_interleave(torch.arange(n, device=DEV), new.long())
    at = torch.arange(total, device=DEV) - (torch.cumsum(new.long(), 0) - new.long())[seq]
    position = first[seq] + at
    blocks = (start + case["hi"]) // page + 1
    # the pages that the step writes; the others of a long context are not kept here
    low, high = first // page, (first + new.long() - 1) // page
    each = case["hi"] // page + 2
    pages = torch.randperm(n * each, device=DEV, generator=g).view(n, each)
    column = torch.arange(blocks, device=DEV).view(1, -1)
    mine = (column >= low.view(-1, 1)) & (column <= high.view(-1, 1))
    ids = pages.gather(1, (column - low.view(-1, 1)).clamp(0, each - 1))
    tables = torch.empty(n, blocks, dtype=torch.int32, device=DEV)
    tables[slots] = torch.where(mine, ids, -1).to(torch.int32)
    return slots[seq].to(torch.int32), position.to(torch.int32), tables, n * each


def _frequencies(case):
    """Radians per position of each rotated pair, and the factor on the rotated pairs."""
    r, kind = case["rot"], case["scaling"]
    base, factor, length = 10000.0, 8.0, 8192
    if kind == "base":
        base = base * factor ** (r / (r - 2))
    f = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if kind == "linear":
        f = [v / factor for v in f]
    if kind == "ramp":
        at = [r * math.log(length / (2 * math.pi * turns)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), r - 1)
        far = [min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in range(r // 2)]
        f = [v / factor * w + v * (1 - w) for v, w in zip(f, far)]
    if kind == "bands":
        turns = [length * v / (2 * math.pi) for v in f]
        near = [min(max((t - 1.0) / (4.0 - 1.0), 0.0), 1.0) for t in turns]
        f = [v / factor * (1 - w) + v * w for v, w in zip(f, near)]
    return f, 0.1 * math.log(factor) + 1.0 if kind == "ramp" else 1.0


def _prepare_rope(case, g):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    ids, positions, tables, pages = _rows(case, g)
    n = ids.numel()
    dtype = TYPE[case["x"]]
    if case["packed"]:
        qkv = _normal((n, hq + 2 * hkv, d), dtype, g)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        q, k, v = (_normal((n, h, d), dtype, g) for h in (hq, hkv, hkv))
    f, magnitude = _frequencies(case)
    st = {"case": case, "q": q, "k": k, "v": v, "ids": ids, "positions": positions, "tables": tables,
          "q_out": torch.zeros(n, hq, d, dtype=dtype, device=DEV),
          "k_pool": torch.zeros(pages, hkv, case["page"], d, dtype=TYPE[case["kv"]], device=DEV),
          "v_pool": torch.zeros(pages, hkv, case["page"], d, dtype=TYPE[case["kv"]], device=DEV),
          "f": torch.tensor(f, dtype=torch.float64, device=DEV), "magnitude": magnitude}
    if own:
        st["pa"] = pa = _library()
        sc = SCALE if case["kv"] == "e4m3" else 1.0
        st["pool"] = pa.Pool(st["k_pool"], st["v_pool"], sc, sc)
        more = {"none": {}, "linear": {"factor": 8.0}, "base": {"factor": 8.0},
                "ramp": {"factor": 8.0, "original_positions": 8192, "low": 1.0, "high": 32.0},
                "bands": {"factor": 8.0, "original_positions": 8192, "low": 1.0, "high": 4.0}}[case["scaling"]]
        st["rope"] = pa.Rope(case["rot"], layout=case["layout"], base=10000.0,
                             scaling=None if case["scaling"] == "none" else case["scaling"], **more)
    return st


def _prepare_prompt(case, g):
    n, hq, hkv, d = case["seqs"], case["hq"], case["hkv"], case["d"]
    lengths = _spread(case, g).long()
    ends = torch.cumsum(lengths, 0)
    rows = int(ends[-1]) + case["pad"]
    if case["packed"]:
        qkv = _normal((rows, hq + 2 * hkv, d), torch.bfloat16, g)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        q, k, v = (_normal((rows, h, d), torch.bfloat16, g) for h in (hq, hkv, hkv))
    starts = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), ends]).to(torch.int32)
    st = {"case": case, "q": q, "k": k, "v": v, "starts": starts, "rows": rows,
          "out": torch.zeros(rows, hq, d, dtype=torch.bfloat16, device=DEV)}
    if own:
        st["pa"] = pa = _library()
        st["ws"] = torch.zeros(pa.prompt_workspace_bytes(rows, n, hq, hkv, d), dtype=torch.uint8, device=DEV)
    return st


def _prepare_append4(case, g):
    hkv, d, page = case["hkv"], case["d"], case["page"]
    ids, positions, tables, pages = _rows(case, g)
    n = ids.numel()
    st = {"case": case, "k": _normal((n, hkv, d), TYPE[case["x"]], g), "v": _normal((n, hkv, d), TYPE[case["x"]], g),
          "ids": ids, "positions": positions, "tables": tables,
          "k_codes": torch.zeros(pages, hkv, page, d // 2, dtype=torch.uint8, device=DEV),
          "v_codes": torch.zeros(pages, hkv, page, d // 2, dtype=torch.uint8, device=DEV),
          "k_ranges": torch.zeros(pages, hkv, page, 2, dtype=torch.float16, device=DEV),
          "v_ranges": torch.zeros(pages, hkv, page, 2, dtype=torch.float16, device=DEV),
          "k_out": torch.zeros(n, hkv, d, dtype=torch.float32, device=DEV),
          "v_out": torch.zeros(n, hkv, d, dtype=torch.float32, device=DEV)}
    if own:
        st["pa"] = pa = _library()
        st["pool"] = pa.Pool(st["k_codes"], st["v_codes"], k_ranges=st["k_ranges"], v_ranges=st["v_ranges"])
    return st


def _prepare_attend4(case, g):
    n, hkv, d, page = case["seqs"], case["hkv"], case["d"], case["page"]
    lengths = _whole(n, case["lo"], case["hi"], g)
    blocks = -(-case["hi"] // page)
    pages = n * blocks
    tables = torch.randperm(pages, device=DEV, generator=g).view(n, blocks).to(torch.int32)
    st = {"case": case, "q": _normal((n, case["hq"], d), TYPE[case["x"]], g), "tables": tables,
          "ids": torch.randperm(n, device=DEV, generator=g).to(torch.int32), "positions": lengths - 1}
    for name in ("k", "v"):
        st[name + "_codes"] = torch.randint(0, 256, (pages, hkv, page, d // 2), device=DEV, generator=g,
                                            dtype=torch.uint8)
        # the ranges of 4-bit codes of about N(0, 1) values
        step = torch.empty(pages, hkv, page, device=DEV).uniform_(0.2, 0.4, generator=g)
        low = step * torch.empty_like(step).uniform_(-9.0, -6.0, generator=g)
        st[name + "_ranges"] = torch.stack([step, low], dim=3).to(torch.float16)
    st["out"] = torch.zeros_like(st["q"])
    if own:
        st["pa"] = pa = _library()
        st["pool"] = pa.Pool(st["k_codes"], st["v_codes"], k_ranges=st["k_ranges"], v_ranges=st["v_ranges"])
        size = pa.workspace_bytes(st["pool"], n, case["hq"], blocks)
        st["ws"] = torch.zeros(size, dtype=torch.uint8, device=DEV) if size else None
    return st


# -------------------------------------------------------------------- run --

def run(state):
    op = state["case"]["op"]
    if own:
        return {"tables": _own_tables, "rope": _own_rope, "prompt": _own_prompt, "append4": _own_append4,
                "attend4": _own_attend4}[op](state)
    return {"tables": _plain_tables, "rope": _plain_rope, "prompt": _plain_prompt, "append4": _plain_append4,
            "attend4": _plain_attend4}[op](state)


def _stored(pool):
    """A pool as the values that its codes stand for, up to its scale."""
    return pool.view(torch.float8_e4m3fn) if pool.dtype == torch.uint8 else pool


def _tables_out(st):
    return tuple(st[name] for name in ("tables", "row_starts", "page_starts", "row_seqs", "row_positions", "row_slots",
                                       "left"))


def _own_tables(st):
    st["pa"].tables_grow(st["seqs"], st["lengths"], st["new"], st["free"], st["count"], st["left"], st["case"]["page"],
                         st["tables"], st["row_starts"], st["page_starts"], st["row_seqs"], st["row_positions"],
                         row_slots=st["row_slots"])
    return _tables_out(st)


def _own_rope(st):
    st["pa"].rope_append(st["pool"], st["rope"], st["q"], st["k"], st["v"], st["ids"], st["positions"], st["tables"],
                         st["q_out"])
    return st["q_out"], _stored(st["k_pool"]), _stored(st["v_pool"])


def _own_prompt(st):
    st["pa"].prompt_attention(st["q"], st["k"], st["v"], st["starts"], st["out"], workspace=st["ws"])
    return st["out"]


def _own_append4(st):
    st["pa"].append_kv(st["pool"], st["k"], st["v"], st["ids"], st["positions"], st["tables"])
    st["pa"].read_kv(st["pool"], st["ids"], st["positions"], st["tables"], st["k_out"], st["v_out"])
    return st["k_out"], st["v_out"]


def _own_attend4(st):
    st["pa"].attention(st["pool"], st["q"], st["ids"], st["positions"], st["tables"], st["out"], workspace=st["ws"])
    return st["out"]


def _plain_tables(st):
    page = st["case"]["page"]
    lengths, new, seqs = st["lengths"].long(), st["new"].long(), st["seqs"].long()
    held = (lengths + page - 1) // page
    need = (lengths + new + page - 1) // page - held
    st["row_starts"][1:] = torch.cumsum(new, 0)
    st["page_starts"][1:] = torch.cumsum(need, 0)
    request = torch.repeat_interleave(torch.arange(need.numel(), device=DEV), need)
    taken = torch.arange(request.numel(), device=DEV)
    column = held[request] + taken - (torch.cumsum(need, 0) - need)[request]
    st["tables"][seqs[request], column] = st["free"][st["count"].long() - 1 - taken]
    st["left"].copy_(st["count"] - st["page_starts"][-1])
    row = torch.repeat_interleave(torch.arange(new.numel(), device=DEV), new)
    position = lengths[row] + torch.arange(row.numel(), device=DEV) - (torch.cumsum(new, 0) - new)[row]
    st["row_seqs"][:row.numel()] = st["seqs"][row]
    st["row_positions"][:row.numel()] = position.to(torch.int32)
    at = st["tables"][seqs[row], position // page].long()
    st["row_slots"][:row.numel()] = at * page + position % page
    return _tables_out(st)


def _rotated(x, st):
    """Rows [n, heads, d] as 32-bit values, rotated; angles of far positions in 64 bits."""
    case = st["case"]
    r = case["rot"]
    angle = st["positions"].double().view(-1, 1, 1) * st["f"]
    cos, sin = (angle.cos() * st["magnitude"]).float(), (angle.sin() * st["magnitude"]).float()
    y = x.float()
    out = y.clone()
    if case["layout"] == "half":
        a, b = y[:, :, :r // 2], y[:, :, r // 2:r]
        out[:, :, :r // 2], out[:, :, r // 2:r] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = y[:, :, 0:r:2], y[:, :, 1:r:2]
        out[:, :, 0:r:2], out[:, :, 1:r:2] = a * cos - b * sin, a * sin + b * cos
    return out


def _stored_as(x, kv):
    if kv == "e4m3":
        return (x / SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return x.to(TYPE[kv])


def _plain_rope(st):
    case = st["case"]
    page = case["page"]
    position = st["positions"].long()
    at, slot = st["tables"][st["ids"].long(), position // page].long(), position % page
    st["q_out"].copy_(_rotated(st["q"], st))
    st["k_pool"][at, :, slot] = _stored_as(_rotated(st["k"], st), case["kv"])
    st["v_pool"][at, :, slot] = _stored_as(st["v"].float(), case["kv"])
    return st["q_out"], _stored(st["k_pool"]), _stored(st["v_pool"])


def _plain_prompt(st):
    case = st["case"]
    n, hkv, d = case["seqs"], case["hkv"], case["d"]
    group = case["hq"] // hkv
    starts = st["starts"].long()
    lengths = starts[1:] - starts[:-1]
    most = case["hi"]
    # every prompt padded to the longest
    token = torch.arange(most, device=DEV)
    rows = (starts[:-1].view(n, 1) + token).clamp(max=st["rows"] - 1)
    q = st["q"][rows].float().view(n, most, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, group * most, d)
    k, v = (st[name][rows].float().transpose(1, 2) for name in ("k", "v"))
    s = torch.matmul(q, k.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).view(n, hkv, group, most, most)
    s.masked_fill_(token.view(1, -1) > token.view(-1, 1), float("-inf"))
    s.sub_(s.amax(dim=4, keepdim=True)).exp_()
    total = s.sum(dim=4, keepdim=True)
    o = torch.matmul(s.view(n, hkv, group * most, most), v).view(n, hkv, group, most, d) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(n, most, case["hq"], d)
    real = token < lengths.view(n, 1)
    st["out"][rows[real]] = o[real].to(st["out"].dtype)
    return st["out"]


def _coded(x):
    """4-bit codes in pairs, and (step, low) in 16 bits, of rows of 32-bit values."""
    x = x.clamp(-65504.0, 65504.0)
    low = x.amin(dim=2, keepdim=True).half()
    step = ((x.amax(dim=2, keepdim=True) - low.float()) / 15.0).half()
    wide = torch.where(step > 0, step.float(), 1.0)
    code = torch.round((x - low.float()) / wide).clamp(0, 15)
    code = torch.where(step > 0, code, 0.0).to(torch.uint8)
    return code[:, :, 0::2] | (code[:, :, 1::2] << 4), torch.cat([step, low], dim=2)


def _values(codes, ranges):
    """What rows of paired codes stand for."""
    code = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).float()
    return code * ranges[..., :1].float() + ranges[..., 1:].float()


def _plain_append4(st):
    page = st["case"]["page"]
    position = st["positions"].long()
    at, slot = st["tables"][st["ids"].long(), position // page].long(), position % page
    for name in ("k", "v"):
        codes, ranges = _coded(st[name].float())
        st[name + "_codes"][at, :, slot], st[name + "_ranges"][at, :, slot] = codes, ranges
        st[name + "_out"].copy_(_values(st[name + "_codes"][at, :, slot], st[name + "_ranges"][at, :, slot]))
    return st["k_out"], st["v_out"]


def _plain_attend4(st):
    case = st["case"]
    n, hkv, d = case["seqs"], case["hkv"], case["d"]
    pages = st["tables"][st["ids"].long()].long()
    k, v = (_values(st[name + "_codes"][pages], st[name + "_ranges"][pages]).transpose(1, 2).reshape(n, hkv, -1, d)
            for name in ("k", "v"))
    q = st["q"].float().view(n, hkv, case["hq"] // hkv, d)
    s = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    s = s.masked_fill(torch.arange(s.shape[3], device=DEV) > st["positions"].view(n, 1, 1, 1), float("-inf"))
    p = torch.exp(s - s.amax(dim=3, keepdim=True))
    o = torch.matmul(p, v) / p.sum(dim=3, keepdim=True)
    st["out"].copy_(o.reshape(n, case["hq"], d))
    return st["out"]


# ------------------------------------------------------------------- work --

def work(case):
    op, n = case["op"], case["seqs"]
    mean = (case["lo"] + case["hi"]) / 2 if n > 1 else case["hi"]
    if op == "tables":
        rows = n * (case["new_lo"] + case["new_hi"]) / 2
        pages = rows / case["page"]
        return {"bytes": 12.0 * n + 8 * pages + 16 * rows + 8 * n, "flops": 0}
    if op == "rope":
        rows, x, kv = n * mean, SIZE[case["x"]], SIZE[case["kv"]]
        moved = case["hq"] * 2 * x + 2 * case["hkv"] * (x + kv)
        return {"bytes": rows * (moved * case["d"] + 12), "flops": 3.0 * rows * (case["hq"] + case["hkv"]) * case["rot"]}
    if op == "prompt":
        # the mean of l (l + 1) / 2 over lengths spread evenly over lo..hi
        lo, hi = case["lo"] if n > 1 else case["hi"], case["hi"]
        pairs = n * ((hi * hi + hi * lo + lo * lo) / 3 + mean) / 2
        return {"bytes": 4.0 * n * mean * (case["hq"] + case["hkv"]) * case["d"],
                "flops": 4.0 * pairs * case["hq"] * case["d"]}
    if op == "append4":
        rows = n * mean * case["hkv"] * 2
        # stored once, and read back into 32 bits
        return {"bytes": rows * (case["d"] * (SIZE[case["x"]] + 4) + 2 * (case["d"] / 2 + 4)), "flops": 4.0 * rows * case["d"]}
    return {"bytes": n * (mean * case["hkv"] * (case["d"] + 8) + 2 * case["hq"] * case["d"] * SIZE[case["x"]]),
            "flops": 4.0 * n * mean * case["hq"] * case["d"]}


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    st = prepare(case, seed)
    return {"tables": lambda c, s: None, "rope": _exact_rope, "prompt": _exact_prompt, "append4": _exact_append4,
            "attend4": _exact_attend4}[case["op"]](case, st)


def _exact_rope(case, st):
    """Each pair as a complex number, turned."""
    r, half = case["rot"], case["layout"] == "half"
    turn = torch.polar(torch.full_like(st["f"], st["magnitude"]) * torch.ones_like(st["positions"]).double().view(-1, 1),
                       torch.outer(st["positions"].double(), st["f"]))

    def turned(x):
        x = x.double()
        pairs = x[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2) if half else x[..., :r].unflatten(-1, (r // 2, 2))
        y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn.unsqueeze(1))
        y = y.transpose(-1, -2).flatten(-2) if half else y.flatten(-2)
        return torch.cat([y, x[..., r:]], dim=-1)

    pools = []
    row = torch.arange(st["ids"].numel(), device=DEV)
    for pool, x in ((st["k_pool"], turned(st["k"])), (st["v_pool"], st["v"].double())):
        new = _stored(pool).float().double()
        page = st["tables"][st["ids"].long(), torch.div(st["positions"], case["page"], rounding_mode="floor").long()]
        new[page.long(), :, st["positions"].long() % case["page"]] = x[row] / (SCALE if case["kv"] == "e4m3" else 1.0)
        pools.append(new)
    return turned(st["q"]), pools[0], pools[1]


def _exact_prompt(case, st):
    out = st["out"].double()
    starts = st["starts"].tolist()
    group = case["hq"] // case["hkv"]
    for a, b in zip(starts[:-1], starts[1:]):
        for h in range(case["hq"]):
            q, k, v = st["q"][a:b, h].double(), st["k"][a:b, h // group].double(), st["v"][a:b, h // group].double()
            for i in range(0, b - a, 2048):
                j = min(b - a, i + 2048)
                s = q[i:j] @ k[:j].T / math.sqrt(case["d"])
                s = s + torch.full_like(s, float("-inf")).triu(i + 1)
                out[a + i:a + j, h] = torch.softmax(s, dim=1) @ v[:j]
    return out


def _exact_append4(case, st):
    """The format's own steps, which are defined in 16 and 32 bits, by numpy; the values in 64."""
    out = []
    for name in ("k", "v"):
        x = np.clip(st[name].float().cpu().numpy(), np.float32(-65504), np.float32(65504))
        low = x.min(axis=2, keepdims=True).astype(np.float16)
        step = ((x.max(axis=2, keepdims=True) - low.astype(np.float32)) / np.float32(15)).astype(np.float16)
        with np.errstate(divide="ignore", invalid="ignore"):
            code = np.rint((x - low.astype(np.float32)) / step.astype(np.float32))
        code = np.where(step == 0, 0, np.minimum(np.maximum(code, 0), 15))
        out.append(torch.from_numpy(code.astype(np.float64) * step.astype(np.float64) + low.astype(np.float64)).to(DEV))
    return tuple(out)


def _exact_attend4(case, st):
    n, hkv, d, page = case["seqs"], case["hkv"], case["d"], case["page"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    for i, (seq, last) in enumerate(zip(st["ids"].tolist(), st["positions"].tolist())):
        ids = st["tables"][seq, :last // page + 1].long()

        def cache(name):
            codes = st[name + "_codes"][ids].transpose(0, 1).reshape(hkv, -1, d // 2)[:, :last + 1]
            pair = st[name + "_ranges"][ids].transpose(0, 1).reshape(hkv, -1, 2)[:, :last + 1].double()
            x = torch.empty(hkv, last + 1, d, dtype=torch.float64, device=DEV)
            x[:, :, 0::2], x[:, :, 1::2] = codes % 16, codes // 16
            return x * pair[:, :, :1] + pair[:, :, 1:]

        q = st["q"][i].double().view(hkv, -1, d)
        s = torch.softmax(q @ cache("k").transpose(1, 2) / math.sqrt(d), dim=2)
        out[i] = (s @ cache("v")).view(-1, d)
    return out
