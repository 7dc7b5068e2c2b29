"""64-bit references of the serving operators (tables, rotary positions, prompt
attention, the 4-bit cache), written from their definitions."""
from __future__ import annotations

import math

import torch

HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def encode4(x):
    """(codes 0..15, step f16, low f16) of rows [..., D], by the format's own steps."""
    x = x.float()
    nan = torch.isnan(x).any(dim=-1, keepdim=True)
    x = torch.nan_to_num(x, nan=0.0, posinf=65504.0, neginf=-65504.0).clamp(-65504.0, 65504.0)
    low = x.amin(dim=-1, keepdim=True).half()
    step = ((x.amax(dim=-1, keepdim=True) - low.float()) / 15.0).clamp(min=0.0).half()
    code = torch.round((x - low.float()) / torch.where(step > 0, step.float(), 1.0)).clamp(0, 15)
    code = torch.where((step > 0) & ~nan, code, 0.0)
    bad = torch.full_like(low, float("nan"))
    return code.to(torch.uint8), torch.where(nan, bad, step), torch.where(nan, bad, low)


def values4(codes, ranges):
    """float64 values of packed codes [..., D / 2] and pairs [..., 2]."""
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).double()
    return c * ranges[..., :1].double() + ranges[..., 1:].double()


def pack4(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def rotate(x, positions, f, magnitude, rot, interleaved, inverse=False):
    """float64 rotated rows [n, heads, D], and the size |a| + |b| of each element's pair."""
    x = x.double()
    angle = positions.double().view(-1, 1, 1) * torch.as_tensor(f, dtype=torch.float64, device=x.device)
    c, s = angle.cos() * magnitude, angle.sin() * magnitude * (-1.0 if inverse else 1.0)
    out, size = x.clone(), torch.zeros_like(x)
    i = torch.arange(rot // 2, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    a, b = x[:, :, ia], x[:, :, ib]
    out[:, :, ia], out[:, :, ib] = a * c - b * s, a * s + b * c
    size[:, :, ia] = size[:, :, ib] = (a.abs() + b.abs()) * magnitude
    return out, size


def rotate_bound(size, out, dtype):
    """The angle in FP32 half turns is off by 2^-25 (a quarter of a turn's sine by pi 2^-25),
    sincospi by 2 units of 2^-24, the magnitude, the products and the sum by 2^-24 each: below
    2^-21 of the pair's size in all; then the rounding to dtype."""
    return 2.0 ** -21 * size + HALF_STEP[dtype] * (out.abs() + 2.0 ** -21 * size) + 1e-38


def causal(q, k, v, scale):
    """float64 causal attention of one sequence: out, sum of p |v|, log-sum-exp, the largest
    sum of |q k| scale."""
    n, hq, d = q.shape
    g = hq // k.shape[1]
    q, k, v = (x.double().transpose(0, 1) for x in (q, k, v))
    k, v = k.repeat_interleave(g, 0), v.repeat_interleave(g, 0)
    big = float((q.abs() @ k.abs().transpose(1, 2)).max()) * scale
    s = (q @ k.transpose(1, 2)) * scale
    s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device=q.device).triu(1), float("-inf"))
    p = torch.softmax(s, dim=2)
    return (p @ v).transpose(0, 1), (p @ v.abs()).transpose(0, 1), torch.logsumexp(s, dim=2).transpose(0, 1), big


def score_error(d, big):
    """A score is an FP32 sum of d products (tensor cores may truncate: 2^-23 a step) of sizes
    that add up to `big`, with a few roundings beside."""
    return (d + 16) * 2.0 ** -23 * big


def causal_bound(out, size, d, n, big):
    """Weights rounded to bf16 (2^-8), scores off by score_error in numerator and denominator,
    ex2 twice 2^-22, sums of n terms and accumulators truncated at each step, the output's rounding."""
    rel = 2.0 ** -8 + 2 * score_error(d, big) + 2.0 ** -21 + (n + 8) * 2.0 ** -23
    return rel * size + 2.0 ** -8 * (out.abs() + rel * size) + 1e-30


def attend4(q, k, v, scale):
    """One row over float64 values k, v [Hkv, T, D]: out, sum of p |v|."""
    hkv = k.shape[0]
    qd = q.double().view(hkv, -1, q.shape[-1])
    p = torch.softmax(qd @ k.transpose(1, 2) * scale, dim=2)
    return (p @ v).reshape(q.shape), p


def attend4_bound(q, out, p, k_ranges, v_ranges, scale):
    """A score is step (q . c) + low sum(q), terms that add up to (47 step + |low|) sum |q| and less.  A
    row's query is f16 after scaling by a power of two: bf16 numbers are exact down to 2^-27 of its
    largest element, f32 ones two parts (2^-22, one unit of score_error's).
    A weight w = p step multiplies c - 8, in -8..7: f16 (2^-11) for bf16 rows, two parts (2^-22) for f32
    ones; the f16 grid of 2^-24 is 2^-30 of the largest weight, below a unit of the sums' 2^-23.
    p (low + 8 step) is FP32.  Sums of T terms, truncated at 2^-23 a step.  The output's rounding."""
    hkv, t = k_ranges.shape[:2]
    d = q.shape[-1]
    qd = q.double().view(hkv, -1, d)
    step, low = k_ranges[..., 0].double(), k_ranges[..., 1].double()
    big = float(((47 * step + low.abs()).unsqueeze(1) * qd.abs().sum(dim=2, keepdim=True)).max()) * scale
    vs, vl = v_ranges[..., 0].double(), v_ranges[..., 1].double()
    size = (p @ (8 * vs + (vl + 8 * vs).abs()).unsqueeze(2)).expand(-1, -1, d).reshape(q.shape)
    rel = 2.0 ** -11 if q.dtype == torch.bfloat16 else 2.0 ** -22
    rel += 2 * score_error(d, big) + 2.0 ** -21 + (t + 8) * 2.0 ** -23
    return rel * size + HALF_STEP[q.dtype] * (out.abs() + rel * size) + 1e-30


def grow(seq_ids, lengths, new, free, count, page, tables, max_rows):
    """pa_tables_grow in plain Python on lists: (tables, row_starts, page_starts, rows, left, status)."""
    num_seqs, blocks = len(tables), len(tables[0])
    tables = [list(r) for r in tables]
    status = 0
    asked_rows = asked_pages = 0
    row_starts, page_starts, rows = [0], [0], []
    for s, length, more in zip(seq_ids, lengths, new):
        ok = 0 <= s < num_seqs and seq_ids.count(s) == 1 and length >= 0 and more >= 0 and length + more <= blocks * page
        need = -(-(length + more) // page) - -(-length // page) if ok else 0
        want = more if ok else 0
        if not ok:
            status = status or 3
        asked_rows, asked_pages = asked_rows + want, asked_pages + need
        served = asked_rows <= max_rows and asked_pages <= count
        if want and not served:
            status = status or 6
        if ok and served:
            for c in range(need):
                tables[s][-(-length // page) + c] = free[count - 1 - page_starts[-1] - c]
            rows += [(s, length + i, tables[s][(length + i) // page] * page + (length + i) % page) for i in range(more)]
            row_starts.append(row_starts[-1] + more)
            page_starts.append(page_starts[-1] + need)
        else:
            row_starts.append(row_starts[-1])
            page_starts.append(page_starts[-1])
    return tables, row_starts, page_starts, rows, count - page_starts[-1], status


def scale_of(d):
    return 1.0 / math.sqrt(d)
