"""The cache operators around paged attention, as cases to be measured.

Five operators that decide which keys of a paged K/V pool live on and move
them there:

  mass      attention weight that every cached key receives from a step's
            queries, summed over the rows and the query heads of its kv head
            and added to a buffer [sequences, kv heads, tokens]
  select    per sequence and kv head, the `budget` tokens with the most
            accumulated weight (first and last tokens protected)
  compact   the kept tokens' K, V and weight moved to the front of a sequence
  beams     beam search's choice over beams x vocabulary from raw logits
  reorder   the beams' block tables, partial pages and state rows permuted to
            their parents

With ``own`` false, run() computes them in elementary torch operations; with
``own`` true it makes the library's calls.  Sizes are those of this
repository's workloads (batched decode: 512 sequences of 64..2662 tokens, 16
query and 8 kv heads of 128; long context: 32768 tokens, 32 query heads; pages
of 16 to 256 tokens) or generic ones.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
KV = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.uint8}
ELT = {"f32": 4, "bf16": 2, "e4m3": 1}


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # a few short conversations: the call's latency is what counts
        {"name": "mass 4 rows short", "op": "mass", "rows": 4, "window": 1, "lo": 64, "hi": 900, "hq": 16, "hkv": 8,
         "d": 128, "page": 32, "kv": "bf16", "q": "bf16"},
        # the batched decode step: one query per sequence, ragged lengths
        {"name": "mass 512 rows ragged", "op": "mass", "rows": 512, "window": 1, "lo": 64, "hi": 2662, "hq": 16,
         "hkv": 8, "d": 128, "page": 32, "kv": "bf16", "q": "bf16"},
        # long contexts in an fp8 cache, where eviction pays most
        {"name": "mass 32 rows long fp8", "op": "mass", "rows": 32, "window": 1, "lo": 30000, "hi": 32768, "hq": 32,
         "hkv": 8, "d": 128, "page": 16, "kv": "e4m3", "q": "bf16"},
        # the last 64 queries of eight prompts vote on the prompt's keys
        {"name": "mass 64-row windows", "op": "mass", "rows": 8, "window": 64, "lo": 4000, "hi": 16384, "hq": 32,
         "hkv": 8, "d": 128, "page": 64, "kv": "bf16", "q": "bf16"},
        # a small batch reaches its budget
        {"name": "select 256 of 900", "op": "select", "seqs": 4, "hkv": 8, "lo": 300, "hi": 900, "budget": 256,
         "first": 4, "last": 32},
        # long contexts cut to a sixteenth
        {"name": "select 2048 of 32768", "op": "select", "seqs": 64, "hkv": 8, "lo": 30000, "hi": 32768,
         "budget": 2048, "first": 4, "last": 256},
        # a small batch's pages closed up in place
        {"name": "compact 8 small", "op": "compact", "seqs": 8, "hkv": 8, "d": 128, "page": 32, "kv": "bf16",
         "lo": 300, "hi": 900, "budget": 256, "copy": False},
        # a large batch cut to an eighth in place
        {"name": "compact 64 large", "op": "compact", "seqs": 64, "hkv": 8, "d": 128, "page": 32, "kv": "bf16",
         "lo": 6000, "hi": 8192, "budget": 1024, "copy": False},
        # one request, four beams
        {"name": "beams 1x4", "op": "beams", "groups": 1, "beams": 4, "vocab": 32000, "pad": 0, "out": 8,
         "dtype": "bf16"},
        # a full batch with a large vocabulary and float logits
        {"name": "beams 64x8 f32", "op": "beams", "groups": 64, "beams": 8, "vocab": 131071, "pad": 1, "out": 16,
         "dtype": "f32"},
        # one request's four beams between two steps
        {"name": "reorder 1x4", "op": "reorder", "groups": 1, "beams": 4, "hkv": 8, "d": 128, "page": 32,
         "kv": "bf16", "lo": 700, "hi": 700, "state": 0},
        # a full batch of beams, with a row of float state for each
        {"name": "reorder 64x8", "op": "reorder", "groups": 64, "beams": 8, "hkv": 8, "d": 128, "page": 64,
         "kv": "bf16", "lo": 300, "hi": 1000, "state": 8192},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["mass", "mass", "select", "compact", "beams", "reorder"])
    kv = rng.choice(["bf16", "bf16", "e4m3", "f32"])
    page = rng.choice([16, 32, 64, 128, 256])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    if op == "mass":
        group = rng.randint(1, 8)
        window = rng.choice([1, 1, _log(rng, 2, 512)])
        hi = _log(rng, max(64, window), 32768)
        # no more keys in all than the largest listed case reads
        rows = max(1, min(_log(rng, 1, 512), 32 * 32768 * 8 // (hi * hkv)))
        if window > 1:
            rows = max(1, min(rows, 16, 8 * 16384 * 32 * 64 // (window * group * hkv * hi)))
        return {"op": op, "rows": rows, "window": window, "lo": max(window, hi // 4, 1), "hi": hi,
                "hq": group * hkv, "hkv": hkv, "d": d, "page": page, "kv": kv, "q": rng.choice(["bf16", "bf16", "f32"])}
    if op == "select":
        hi = _log(rng, 1, 131072)
        budget = min(_log(rng, 1, 4096), max(1, hi))
        first, last = (rng.randint(0, budget // 4), rng.randint(0, budget // 2))
        return {"op": op, "seqs": max(1, min(_log(rng, 1, 256), 64 * 32768 * 8 // (hi * hkv))), "hkv": hkv,
                "lo": max(1, hi // 3), "hi": hi, "budget": budget, "first": first, "last": last}
    if op == "compact":
        hi = _log(rng, 16, 16384)
        budget = min(_log(rng, 1, 4096), hi)
        row = hkv * d * ELT[kv]
        most = min(64 * 8192 * 2048 // (hi * row), 64 * 1024 * 2048 // (budget * row))
        return {"op": op, "seqs": max(1, min(_log(rng, 1, 128), most)), "hkv": hkv, "d": d, "page": page, "kv": kv,
                "lo": max(1, hi // 3), "hi": hi, "budget": budget, "copy": rng.random() < 0.4}
    if op == "beams":
        beams = rng.randint(1, 16)
        vocab = _log(rng, 64, 262144)
        groups = max(1, min(_log(rng, 1, 128), 64 * 8 * 131072 // (beams * vocab)))
        return {"op": op, "groups": groups, "beams": beams, "vocab": vocab, "pad": rng.choice([0, 0, 3, 8]),
                "out": rng.randint(1, 2 * beams), "dtype": rng.choice(["bf16", "f32"])}
    beams = rng.randint(1, 16)
    hi = _log(rng, 1, 2000)
    row = hkv * d * ELT[kv]
    groups = max(1, min(_log(rng, 1, 128), 64 * 8 * 64 * 2048 // (beams * page * row),
                        64 * 8 * 1024 * 2048 // (beams * max(hi, page) * row)))
    return {"op": op, "groups": groups, "beams": beams, "hkv": hkv, "d": d, "page": page, "kv": kv, "lo": max(1, hi // 3),
            "hi": hi, "state": rng.choice([0, 0, 257, 4096])}


# ----------------------------------------------------------------- inputs --

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _lengths(n, lo, hi, g):
    return torch.randint(lo, hi + 1, (n,), device=DEV, generator=g, dtype=torch.int32)


def _pool(pages, hkv, page, d, kv, g):
    """Random K or V pages; fp8 ones hold N(0, 1) / scale with scale 1/32."""
    x = torch.empty(pages, hkv, page, d, device=DEV, dtype=torch.float32 if kv == "f32" else torch.bfloat16)
    x.normal_(generator=g)
    if kv == "e4m3":
        x = (x * 32.0).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return x


SCALE = 1.0 / 32.0  # of the fp8 pools


def _tables(num_seqs, blocks, g):
    """Every sequence's pages, in random order over the pool."""
    return torch.randperm(num_seqs * blocks, device=DEV, generator=g).view(num_seqs, blocks).to(torch.int32)


def _handle(st, case):
    if own:
        import paged_kv_continuous_pa_gb300 as pa
        st["pa"] = pa
        if "k" in st:
            sc = SCALE if case["kv"] == "e4m3" else 1.0
            st["pool"] = pa.Pool(st["k"], st["v"], sc, sc)
    return st


def _values(pool):
    """A pool as the values that its codes stand for, up to its scale."""
    return pool.view(torch.float8_e4m3fn) if pool.dtype == torch.uint8 else pool


def prepare(case, seed):
    g = _generator(seed)
    return {"mass": _prepare_mass, "select": _prepare_select, "compact": _prepare_compact, "beams": _prepare_beams,
            "reorder": _prepare_reorder}[case["op"]](case, g)


def _prepare_mass(case, g):
    n, w, hkv = case["rows"], case["window"], case["hkv"]
    lengths = _lengths(n, case["lo"], case["hi"], g)
    blocks = -(-case["hi"] // case["page"])
    tables = _tables(n, blocks, g)
    seqs = torch.randperm(n, device=DEV, generator=g).to(torch.int32)
    k = _pool(n * blocks, hkv, case["page"], case["d"], case["kv"], g)
    q = torch.empty(n * w, case["hq"], case["d"], device=DEV, dtype=KV[case["q"]]).normal_(generator=g)
    mass = torch.empty(n, hkv, blocks * case["page"], device=DEV).exponential_(generator=g)
    # the rows of a window are the last tokens of their sequence, in order
    seq_ids = seqs.repeat_interleave(w)
    positions = (lengths.repeat_interleave(w) - w + torch.arange(w, device=DEV, dtype=torch.int32).repeat(n)).to(torch.int32)
    st = {"case": case, "k": k, "v": k, "q": q, "tables": tables, "seqs": seqs, "seq_ids": seq_ids,
          "positions": positions, "mass": mass, "chunks": [(i * w, w) for i in range(n)] if w > 1 else []}
    _handle(st, case)
    if own:
        size = st["pa"].mass_workspace_bytes(st["pool"], n * w, case["hq"], blocks, st["chunks"])
        st["ws"] = torch.zeros(size, dtype=torch.uint8, device=DEV) if size else None
    return st


def _prepare_select(case, g):
    n, hkv = case["seqs"], case["hkv"]
    lengths = _lengths(n, case["lo"], case["hi"], g)
    # accumulated weight: spread over decades, and zero for keys no query has looked at
    mass = torch.empty(n, hkv, case["hi"], device=DEV).normal_(std=3.0, generator=g).exp_()
    mass.masked_fill_(torch.rand(mass.shape, device=DEV, generator=g) < 0.05, 0.0)
    seqs = torch.randperm(n, device=DEV, generator=g).to(torch.int32)
    st = {"case": case, "mass": mass, "lengths": lengths, "seqs": seqs}
    if own:
        st["keep"] = torch.empty(n, hkv, case["budget"], dtype=torch.int32, device=DEV)
        st["kept"] = torch.empty(n, dtype=torch.int32, device=DEV)
    return _handle(st, case)


def _prepare_compact(case, g):
    n, hkv, budget = case["seqs"], case["hkv"], case["budget"]
    slots = 2 * n if case["copy"] else n
    blocks = -(-case["hi"] // case["page"])
    lengths = _lengths(n, case["lo"], case["hi"], g)
    tables = _tables(slots, blocks, g)
    order = torch.randperm(slots, device=DEV, generator=g).to(torch.int32)
    # a kept set of each (sequence, kv head): `budget` random tokens in order
    noise = torch.rand(n, hkv, case["hi"], device=DEV, generator=g)
    noise.masked_fill_(torch.arange(case["hi"], device=DEV) >= lengths.view(n, 1, 1), 2.0)
    keep = noise.topk(budget, dim=-1, largest=False).indices
    count = torch.minimum(lengths, torch.full_like(lengths, budget)).view(n, 1, 1)
    keep = torch.where(keep < lengths.view(n, 1, 1), keep, torch.full_like(keep, 1 << 30)).sort(dim=-1).values
    keep = torch.where(torch.arange(budget, device=DEV) < count, keep, torch.full_like(keep, -1)).to(torch.int32)
    st = {"case": case, "k": _pool(slots * blocks, hkv, case["page"], case["d"], case["kv"], g),
          "v": _pool(slots * blocks, hkv, case["page"], case["d"], case["kv"], g), "tables": tables,
          "lengths": lengths, "keep": keep, "seqs": order[:n].contiguous(),
          "dst": order[n:].contiguous() if case["copy"] else None,
          "mass": torch.empty(slots, hkv, blocks * case["page"], device=DEV).exponential_(generator=g)}
    return _handle(st, case)


def _prepare_beams(case, g):
    n, b, v = case["groups"], case["beams"], case["vocab"]
    room = torch.empty(n, b, v + case["pad"], device=DEV, dtype=KV[case["dtype"]]).normal_(std=2.5, generator=g)
    logits = room[:, :, :v]
    # some tokens are forbidden, and some beams have ended
    logits.masked_fill_(torch.rand(v, device=DEV, generator=g) < 0.01, float("-inf"))
    scores = -torch.empty(n, b, device=DEV).exponential_(0.2, generator=g)
    finished = (torch.rand(n, b, device=DEV, generator=g) < 0.1).to(torch.int32)
    st = {"case": case, "logits": logits, "scores": scores, "finished": finished}
    if own:
        import paged_kv_continuous_pa_gb300 as pa
        st["out"] = (torch.empty(n, case["out"], dtype=torch.int32, device=DEV),
                     torch.empty(n, case["out"], dtype=torch.int32, device=DEV),
                     torch.empty(n, case["out"], dtype=torch.float32, device=DEV))
        size = pa.beam_workspace_bytes(n, b, v, case["out"])
        st["ws"] = torch.zeros(size, dtype=torch.uint8, device=DEV) if size else None
    return _handle(st, case)


def _prepare_reorder(case, g):
    n, b, page = case["groups"], case["beams"], case["page"]
    blocks = case["hi"] // page + 1  # room for the next token
    lengths = _lengths(n, case["lo"], case["hi"], g)
    own_pages = _tables(n * b, blocks, g)
    # finished pages are any beam's of the group, the rest is each beam's own
    group = torch.arange(n, device=DEV).view(n, 1, 1)
    origin = torch.randint(0, b, (n, b, blocks), device=DEV, generator=g) + group * b
    shared = own_pages[origin, torch.arange(blocks, device=DEV)]
    full = (lengths // page).view(n, 1, 1) > torch.arange(blocks, device=DEV)
    rows = torch.where(full, shared, own_pages.view(n, b, blocks)).view(n * b, blocks)
    seqs = torch.randperm(n * b, device=DEV, generator=g).to(torch.int32)
    tables = torch.empty_like(rows)
    tables[seqs.long()] = rows
    st = {"case": case, "k": _pool(n * b * blocks, case["hkv"], page, case["d"], case["kv"], g),
          "v": _pool(n * b * blocks, case["hkv"], page, case["d"], case["kv"], g), "tables": tables,
          "lengths": lengths, "seqs": seqs.view(n, b),
          "parents": torch.randint(0, b, (n, b), device=DEV, generator=g, dtype=torch.int32),
          "state": torch.empty(n * b, case["state"], device=DEV).normal_(generator=g) if case["state"] else None}
    return _handle(st, case)


# -------------------------------------------------------------------- run --

def run(state):
    op = state["case"]["op"]
    if own:
        return {"mass": _own_mass, "select": _own_select, "compact": _own_compact, "beams": _own_beams,
                "reorder": _own_reorder}[op](state)
    return {"mass": _plain_mass, "select": _plain_select, "compact": _plain_compact, "beams": _plain_beams,
            "reorder": _plain_reorder}[op](state)


def _own_mass(st):
    st["pa"].attention_mass(st["pool"], st["q"], st["seq_ids"], st["positions"], st["tables"], st["mass"],
                            chunks=st["chunks"], workspace=st["ws"])
    return st["mass"]


def _own_select(st):
    st["pa"].evict_select(st["mass"], st["seqs"], st["lengths"], st["keep"], kept_lengths=st["kept"],
                          keep_first=st["case"]["first"], keep_last=st["case"]["last"])
    return st["keep"], st["kept"]


def _own_compact(st):
    st["pa"].evict_compact(st["pool"], st["keep"], st["seqs"], st["lengths"], st["tables"], mass=st["mass"],
                           dst_seq_ids=st["dst"])
    return _values(st["k"]), _values(st["v"]), st["mass"]


def _own_beams(st):
    parents, tokens, scores = st["out"]
    st["pa"].beam_select(st["logits"], st["scores"], parents, tokens, scores, finished=st["finished"], end_token=2,
                         workspace=st["ws"])
    return parents, tokens, scores


def _own_reorder(st):
    st["pa"].beam_reorder(st["pool"], st["parents"], st["seqs"], st["lengths"], st["tables"], state=st["state"])
    out = [st["tables"], _values(st["k"]), _values(st["v"])]
    return out + [st["state"]] if st["state"] is not None else out


def _floats(x, scale):
    """Cached elements as 32-bit values."""
    if x.dtype == torch.uint8:
        return x.view(torch.float8_e4m3fn).float() * scale
    return x.float()


def _plain_mass(st):
    case, n = st["case"], st["case"]["rows"]
    w, hkv, d = case["window"], case["hkv"], case["d"]
    group = case["hq"] // hkv
    pages = st["tables"][st["seqs"].long()].long()
    k = _floats(st["k"][pages].transpose(1, 2).reshape(n, hkv, -1, d), SCALE)
    # the queries that share a kv head, over the rows of a window
    q = st["q"].view(n, w, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, w * group, d).float()
    s = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    keys = torch.arange(s.shape[3], device=DEV)
    last = st["positions"].view(n, 1, w, 1, 1).expand(n, 1, w, group, 1).reshape(n, 1, w * group, 1)
    s = s.masked_fill(keys > last, float("-inf"))
    p = torch.exp(s - s.amax(dim=3, keepdim=True))
    p = p / p.sum(dim=3, keepdim=True)
    st["mass"].index_add_(0, st["seqs"], p.sum(dim=2))
    return st["mass"]


def _descending(x):
    """int64 keys whose order is that of the values, ties by lowest index first."""
    bits = x.contiguous().view(torch.int32).long()
    order = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    return (order << 32) | (0xFFFFFFFF - torch.arange(x.shape[-1], device=x.device))


def _plain_select(st):
    case, mass = st["case"], st["mass"][st["seqs"].long()]
    n, budget = case["seqs"], case["budget"]
    lengths = st["lengths"].long().view(n, 1, 1)
    at = torch.arange(mass.shape[2], device=DEV)
    safe = (at < case["first"]) | (at >= lengths - case["last"])
    value = mass.masked_fill(safe, float("inf")).masked_fill(at >= lengths, float("-inf"))
    best = torch.topk(_descending(value), min(budget, mass.shape[2]), dim=2, sorted=False).indices
    best = best.masked_fill(best >= lengths, 1 << 40).sort(dim=2).values
    keep = torch.full((n, mass.shape[1], budget), -1, dtype=torch.int32, device=DEV)
    keep[:, :, :best.shape[2]] = best.masked_fill(best >= 1 << 40, -1).to(torch.int32)
    return keep, torch.clamp(st["lengths"], max=budget)


def _plain_compact(st):
    case = st["case"]
    page, budget = case["page"], case["budget"]
    src, dst = st["seqs"].long(), (st["seqs"] if st["dst"] is None else st["dst"]).long()
    seq, head, to = torch.nonzero(st["keep"] >= 0, as_tuple=True)
    at = st["keep"][seq, head, to].long()
    from_page, to_page = st["tables"][src[seq], at // page].long(), st["tables"][dst[seq], to // page].long()
    for pool in (st["k"], st["v"]):
        pool[to_page, head, to % page] = pool[from_page, head, at % page]
    moved = st["mass"][src[seq], head, at]
    keys = torch.arange(st["mass"].shape[2], device=DEV)
    lengths = st["lengths"].view(-1, 1)
    emptied = (keys >= lengths.clamp(max=budget)) & (keys < lengths)
    st["mass"][dst] = st["mass"][dst].masked_fill(emptied.unsqueeze(1), 0.0)
    st["mass"][dst[seq], head, to] = moved
    return _values(st["k"]), _values(st["v"]), st["mass"]


def _plain_beams(st):
    case = st["case"]
    n, b, v, out = case["groups"], case["beams"], case["vocab"], case["out"]
    x = st["logits"].float()
    top = x.amax(dim=2, keepdim=True)
    # long sums, and scores of which the nearest decide: 64 bits
    norm = top.double() + torch.log(torch.exp(x - top).sum(dim=2, keepdim=True, dtype=torch.float64))
    at = torch.topk(_descending(x), min(out, v), dim=2).indices
    score = st["scores"].double().unsqueeze(2) + (x.gather(2, at).double() - norm)
    # a beam that has ended goes on as it is
    ended = st["finished"].bool().unsqueeze(2)
    rank = torch.arange(at.shape[2], device=DEV)
    score = torch.where(ended, torch.where(rank == 0, st["scores"].double().unsqueeze(2), float("-inf")), score)
    at = torch.where(ended, 2, at)
    score = torch.where(torch.isfinite(score), score, float("-inf")).view(n, -1)
    best, where = torch.sort(score, dim=1, descending=True, stable=True)
    best, where = best[:, :out], where[:, :out]
    real = best > float("-inf")
    parents = torch.full((n, out), -1, dtype=torch.int32, device=DEV)
    tokens, scores = parents.clone(), torch.full((n, out), float("-inf"), device=DEV)
    parents[:, :where.shape[1]] = torch.where(real, where // at.shape[2], -1).to(torch.int32)
    tokens[:, :where.shape[1]] = torch.where(real, at.reshape(n, -1).gather(1, where), -1).to(torch.int32)
    scores[:, :where.shape[1]] = best.float()
    return parents, tokens, scores


def _plain_reorder(st):
    case = st["case"]
    n, b, page = case["groups"], case["beams"], case["page"]
    seqs, lengths = st["seqs"].long(), st["lengths"].long()
    parents = seqs.gather(1, st["parents"].long())
    blocks = torch.arange(st["tables"].shape[1], device=DEV)
    full = (lengths // page).view(n, 1, 1) > blocks
    rows = torch.where(full, st["tables"][parents], st["tables"][seqs])
    # the slots in use of each beam's unfinished page
    group, beam, slot = torch.nonzero((lengths % page).view(n, 1, 1).expand(n, b, 1) > torch.arange(page, device=DEV),
                                      as_tuple=True)
    column = lengths[group] // page
    to = st["tables"][seqs[group, beam], column].long()
    at = st["tables"][parents[group, beam], column].long()
    for pool in (st["k"], st["v"]):
        pool[to, :, slot] = pool[at, :, slot]
    st["tables"][seqs] = rows
    out = [st["tables"], _values(st["k"]), _values(st["v"])]
    if st["state"] is not None:
        st["state"][seqs] = st["state"][parents]
        out.append(st["state"])
    return out


# ------------------------------------------------------------------- work --

def work(case):
    op = case["op"]
    mean = (case["lo"] + case["hi"]) / 2 if "lo" in case else 0
    if op == "mass":
        keys = case["rows"] * mean
        flops = 2.0 * case["d"] * case["hq"] * case["window"] * (keys - case["rows"] * (case["window"] - 1) / 2)
        read = keys * case["hkv"] * (case["d"] * ELT[case["kv"]] + 8)
        q = case["rows"] * case["window"] * case["hq"] * case["d"] * ELT[case["q"]]
        return {"bytes": read + q, "flops": flops}
    if op == "select":
        return {"bytes": 4.0 * case["seqs"] * case["hkv"] * (mean + case["budget"]), "flops": 0}
    if op == "compact":
        kept = case["seqs"] * case["hkv"] * min(case["budget"], mean)
        gone = case["seqs"] * case["hkv"] * max(0.0, mean - case["budget"])
        return {"bytes": kept * (4 * case["d"] * ELT[case["kv"]] + 12) + 4 * gone, "flops": 0}
    if op == "beams":
        cells = case["groups"] * case["beams"] * case["vocab"]
        return {"bytes": cells * ELT[case["dtype"]] + 12.0 * case["groups"] * case["out"], "flops": 4.0 * cells}
    # reorder: beams that change hands, half a page of slots on average
    moved = case["groups"] * (case["beams"] - 1 or 1)
    tail = case["page"] / 2 if case["lo"] < case["hi"] else case["hi"] % case["page"]
    row = 4.0 * tail * case["hkv"] * case["d"] * ELT[case["kv"]] + 8.0 * (mean // case["page"]) + 8.0 * case["state"]
    return {"bytes": max(1.0, moved * row), "flops": 0}


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    st = prepare(case, seed)
    return {"mass": _exact_mass, "select": _exact_select, "compact": _exact_compact, "beams": _exact_beams,
            "reorder": _exact_reorder}[case["op"]](case, st)


def _exact_cache(st, seq, length, pool, scale):
    """The first `length` cached rows of a sequence, [kv heads, length, d], in 64 bits."""
    page = pool.shape[2]
    ids = st["tables"][seq, : -(-length // page)].long()
    rows = pool[ids]
    rows = rows.view(torch.float8_e4m3fn).float().double() * scale if rows.dtype == torch.uint8 else rows.double()
    return torch.cat(list(rows), dim=1)[:, :length]


def _exact_mass(case, st):
    w, hkv = case["window"], case["hkv"]
    group = case["hq"] // hkv
    mass = st["mass"].double()
    last = st["positions"].tolist()
    for i, seq in enumerate(st["seqs"].tolist()):
        k = _exact_cache(st, seq, last[i * w + w - 1] + 1, st["k"], SCALE)
        for h in range(hkv):
            q = st["q"][i * w:(i + 1) * w, h * group:(h + 1) * group].double()
            s = torch.einsum("wgd,td->wgt", q, k[h]) / math.sqrt(case["d"])
            seen = torch.arange(k.shape[1], device=DEV).view(1, -1) <= st["positions"][i * w:(i + 1) * w].view(w, 1)
            s = torch.where(seen.unsqueeze(1), s, torch.full_like(s, float("-inf")))
            mass[seq, h, : k.shape[1]] += torch.softmax(s, dim=2).sum(dim=(0, 1))
    return mass


def _exact_select(case, st):
    return None  # whole numbers alone


def _exact_compact(case, st):
    k, v, mass = st["k"].clone(), st["v"].clone(), st["mass"].double()
    into = st["seqs"] if st["dst"] is None else st["dst"]
    page, hkv = case["page"], case["hkv"]
    before = st["mass"].double()
    heads = torch.arange(hkv, device=DEV).view(hkv, 1)
    for i, (seq, to, length) in enumerate(zip(st["seqs"].tolist(), into.tolist(), st["lengths"].tolist())):
        count = min(length, case["budget"])
        at = st["keep"][i, :, :count].long()
        slots = torch.arange(count, device=DEV)
        a, b = st["tables"][seq][at // page].long(), st["tables"][to][slots // page].long().expand(hkv, count)
        for new, old in ((k, st["k"]), (v, st["v"])):
            new[b, heads, (slots % page).expand(hkv, count)] = old[a, heads, at % page]
        mass[to, :, count:length] = 0
        mass[to, :, :count] = before[seq].gather(1, at)
    return _values(k), _values(v), mass


def _exact_beams(case, st):
    n, b, out = case["groups"], case["beams"], case["out"]
    scores = torch.full((n, out), float("-inf"), dtype=torch.float64, device=DEV)
    for i in range(n):
        total = torch.log_softmax(st["logits"][i].double(), dim=1) + st["scores"][i].double().view(b, 1)
        done = st["finished"][i].bool()
        total[done] = float("-inf")
        total[done, 2] = st["scores"][i].double()[done]
        best = torch.sort(total.view(-1), descending=True).values[:out]
        scores[i, : best.numel()] = best
    return None, None, scores


def _exact_reorder(case, st):
    k, v, tables = st["k"].clone(), st["v"].clone(), st["tables"].clone()
    state = None if st["state"] is None else st["state"].double()
    page = case["page"]
    for i, length in enumerate(st["lengths"].tolist()):
        whole, tail = divmod(length, page)
        for beam in range(case["beams"]):
            me = int(st["seqs"][i, beam])
            parent = int(st["seqs"][i, int(st["parents"][i, beam])])
            tables[me, :whole] = st["tables"][parent, :whole]
            if tail:
                to, at = int(st["tables"][me, whole]), int(st["tables"][parent, whole])
                k[to, :, :tail], v[to, :, :tail] = st["k"][at, :, :tail], st["v"][at, :, :tail]
            if state is not None:
                state[me] = st["state"][parent].double()
    out = [tables, _values(k), _values(v)]
    return out if state is None else out + [state]
