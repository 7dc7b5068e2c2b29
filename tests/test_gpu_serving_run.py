"""The serving operators as a server runs them: block tables grown on the GPU, projections
rotated and appended, prompts attended to, single tokens decoded in a captured step, pages
given back and handed out again."""
import os
import re

import pytest
import torch

import paged_kv_continuous_pa_gb300 as pa
import serving_ref as R

pytestmark = pytest.mark.gpu
PAGE, BLOCKS, HQ, HKV, D = 16, 24, 8, 2, 64
PROMPTS = [70, 1, 200, 16, 33]
NEW = 20


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def zeros(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


class Server:
    """Requests in slots of one pool; all the state that a step changes is on the GPU."""

    def __init__(self, kind, n, scaling=None):
        pages = n * BLOCKS
        self.kind, self.n = kind, n
        if kind == "int4":
            codes = [zeros(pages, HKV, PAGE, D // 2, dtype=torch.uint8) for _ in "kv"]
            self.ranges = [zeros(pages, HKV, PAGE, 2, dtype=torch.float16) for _ in "kv"]
            self.pool = pa.Pool(*codes, k_ranges=self.ranges[0], v_ranges=self.ranges[1])
        else:
            self.pool = pa.Pool(*[zeros(pages, HKV, PAGE, D, dtype=torch.bfloat16) for _ in "kv"])
        g = torch.Generator().manual_seed(3)
        self.free = torch.randperm(pages, generator=g).to(torch.int32).cuda()
        self.count, self.status = ints([pages]), zeros(1)
        self.tables = torch.full((n, BLOCKS), -1, dtype=torch.int32, device="cuda")
        self.ids, self.lengths = torch.arange(n, dtype=torch.int32, device="cuda"), zeros(n)
        self.rope = pa.Rope(D, scaling=scaling, factor=4.0, original_positions=64)
        size = pa.workspace_bytes(self.pool, n, HQ, BLOCKS, ())
        self.ws = zeros(max(size, 1), dtype=torch.uint8)

    def grow(self, new, rows, ids=None, lengths=None):
        ids, lengths = (self.ids, self.lengths) if ids is None else (ids, lengths)
        n = ids.shape[0]
        out = zeros(n + 1), zeros(n + 1), zeros(rows), zeros(rows), torch.full((rows,), -9, dtype=torch.int64, device="cuda")
        pa.tables_grow(ids, lengths, new, self.free, self.count, self.count, PAGE, self.tables, *out, status=self.status)
        return out

    def take_in(self, qkv, seqs, positions):
        q, k, v = qkv.split([HQ, HKV, HKV], dim=1)
        q_out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
        pa.rope_append(self.pool, self.rope, q, k, v, seqs, positions, self.tables, q_out, status=self.status)
        return q_out

    def prompts(self, lengths, qkv, ids=None, first=None):
        rows = sum(lengths)
        starts, _, seqs, positions, slots = self.grow(ints(lengths), rows, ids, first)
        q = self.take_in(qkv, seqs, positions)
        k, v = zeros(rows, HKV, D, dtype=torch.bfloat16), zeros(rows, HKV, D, dtype=torch.bfloat16)
        pa.read_kv(self.pool, seqs, positions, self.tables, k, v, status=self.status)
        out = torch.empty_like(q)
        ws = zeros(pa.prompt_workspace_bytes(rows, len(lengths), HQ, HKV, D), dtype=torch.uint8)
        pa.prompt_attention(q, k, v, starts, out, workspace=ws, status=self.status)
        return q, k, v, out, starts, seqs, positions, slots

    def decode(self, qkv, out):
        _, _, seqs, positions, _ = self.grow(torch.ones_like(self.lengths), self.n)
        q = self.take_in(qkv, seqs, positions)
        pa.attention(self.pool, q, seqs, positions, self.tables, out, workspace=self.ws, status=self.status)
        self.lengths += 1
        return q

    def cached(self, slot, length):
        """float32 K and V [length, Hkv, D] as read back, and their ranges [Hkv, length, 2] (4-bit pool)."""
        k, v = zeros(length, HKV, D, dtype=torch.float32), zeros(length, HKV, D, dtype=torch.float32)
        t = torch.arange(length, dtype=torch.int32, device="cuda")
        pa.read_kv(self.pool, torch.full_like(t, slot), t, self.tables, k, v, status=self.status)
        if self.kind != "int4":
            return k, v, None
        at = self.tables[slot][t.long() // PAGE].long()
        return k, v, [x[at, :, t.long() % PAGE].transpose(0, 1) for x in self.ranges]


def projections(n, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, HQ + 2 * HKV, D, generator=g).bfloat16().cuda()


def check_row(server, slot, length, q, out):
    """One decoded row against 64-bit attention over what the cache holds (the values as read back:
    one FP32 rounding, less than a unit of the scores' and sums' terms)."""
    k, v, ranges = server.cached(slot, length)
    scale = R.scale_of(D)
    want, p = R.attend4(q, k.double().transpose(0, 1), v.double().transpose(0, 1), scale)
    if ranges is not None:
        bound = R.attend4_bound(q, want, p, *ranges, scale)
    else:
        qd, kd = q.double().view(HKV, -1, D), k.double().transpose(0, 1)
        big = float((qd.abs() @ kd.abs().transpose(1, 2)).max()) * scale
        bound = R.causal_bound(want, (p @ v.double().abs().transpose(0, 1)).reshape(q.shape), D, length, big)
    err = (out.double() - want).abs()
    assert bool((err <= bound).all()), f"slot {slot}, {length} tokens: {float((err / bound).max())} of the bound"


def start(kind, scaling=None):
    s = Server(kind, len(PROMPTS), scaling)
    rows = sum(PROMPTS)
    got = s.prompts(PROMPTS, projections(rows, 1))
    s.lengths += ints(PROMPTS)
    return s, got


@pytest.mark.parametrize("kind,scaling", [("int4", None), ("bf16", None), ("bf16", "ramp")])
def test_prompts_then_captured_decode_steps(kind, scaling):
    s, (q, k, v, out, starts, seqs, positions, slots) = start(kind, scaling)
    at = starts.tolist()
    assert at == [0, 70, 71, 271, 287, 320]
    assert seqs.tolist() == sum(([i] * n for i, n in enumerate(PROMPTS)), [])
    # the prompts' queries and, in a bf16 pool, keys are rotated; their attention is the formula's
    x = projections(sum(PROMPTS), 1)
    f, m = s.rope.frequencies()
    for rows, got in ((x[:, :HQ], q),) + (((x[:, HQ:HQ + HKV], k),) if kind == "bf16" else ()):
        want, size = R.rotate(rows, positions, f, m, D, False)
        assert bool(((got.double() - want).abs() <= R.rotate_bound(size, want, torch.bfloat16)).all())
    if kind == "bf16":
        assert torch.equal(v, x[:, HQ + HKV:])
    for a, b in zip(at, at[1:]):
        want, size, _, big = R.causal(q[a:b], k[a:b], v[a:b], R.scale_of(D))
        err = (out[a:b].double() - want).abs()
        assert bool((err <= R.causal_bound(want, size, D, b - a, big)).all())
    # the tokens' places are those that the tables name
    assert torch.equal(slots, s.tables[seqs.long(), positions.long() // PAGE].long() * PAGE + positions.long() % PAGE)

    # an eager twin takes the same steps
    twin, _ = start(kind, scaling)
    inputs = [projections(len(PROMPTS), 10 + t) for t in range(NEW)]
    qkv, static = inputs[0].clone(), zeros(len(PROMPTS), HQ, D, dtype=torch.bfloat16)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        q_static = s.decode(qkv, static)
    for t in range(NEW):
        qkv.copy_(inputs[t])
        graph.replay()
        eager = torch.empty_like(static)
        q_eager = twin.decode(inputs[t], eager)
        assert torch.equal(static, eager) and torch.equal(q_static, q_eager)
        if t in (0, 14, NEW - 1):
            for i, n in enumerate(PROMPTS):
                check_row(s, i, n + t + 1, q_static[i], static[i])
    assert torch.equal(s.tables, twin.tables) and torch.equal(s.count, twin.count)
    held = sum(-(-(n + NEW) // PAGE) for n in PROMPTS)
    assert s.count.item() == len(PROMPTS) * BLOCKS - held and s.status.item() == 0


def test_pages_given_back_serve_the_next_prompt():
    s, _ = start("int4")
    before, left = s.tables.clone(), s.count.item()
    pa.tables_release(ints([2, 0]), ints([200, 70]), s.free, s.count, PAGE, s.tables, keep_tokens=ints([100, 0]), status=s.status)
    assert s.count.item() == left + (13 - 7) + 5 and s.status.item() == 0
    assert (s.tables[0] == -1).all() and (s.tables[2, 7:] == -1).all() and torch.equal(s.tables[2, :7], before[2, :7])
    # a new request in slot 0, and the one in slot 2 goes on behind the tokens that it kept
    got = s.prompts([50, 9], projections(59, 5), ints([0, 2]), ints([0, 100]))
    assert got[4].tolist() == [0, 50, 59]
    s.lengths.copy_(ints([50, 1, 109, 16, 33]))
    out = zeros(len(PROMPTS), HQ, D, dtype=torch.bfloat16)
    q = s.decode(projections(len(PROMPTS), 6), out)
    for i, n in enumerate([51, 2, 110, 17, 34]):
        check_row(s, i, n, q[i], out[i])
    pages = s.tables[s.tables >= 0].tolist() + s.free[:s.count.item()].tolist()
    assert sorted(pages) == list(range(len(PROMPTS) * BLOCKS)) and s.status.item() == 0


def test_prompts_beside_decode_on_another_stream():
    """Prompts of new requests on a stream of their own, with a workspace of their own, while others decode."""
    s, _ = start("bf16")
    lengths = [700, 129, 257]
    x = projections(sum(lengths), 8)
    q, k, v = (y.contiguous() for y in x.split([HQ, HKV, HKV], dim=1))
    at = ints([0, 700, 829, 1086])
    outs, alone = [torch.empty_like(q) for _ in range(8)], torch.empty_like(q)
    size = pa.prompt_workspace_bytes(q.shape[0], 3, HQ, HKV, D)
    works = [zeros(size, dtype=torch.uint8) for _ in range(2)]
    status = zeros(1)
    pa.prompt_attention(q, k, v, at, alone, workspace=works[0], status=status)
    twin, _ = start("bf16")
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        with torch.cuda.stream(streams[i % 2]):
            pa.prompt_attention(q, k, v, at, out, workspace=works[i % 2], status=status)
    decoded, want = [zeros(len(PROMPTS), HQ, D, dtype=torch.bfloat16) for _ in "ab"]
    for t in range(6):
        s.decode(projections(len(PROMPTS), 40 + t), decoded)
    torch.cuda.synchronize()
    for t in range(6):
        twin.decode(projections(len(PROMPTS), 40 + t), want)
    assert all(torch.equal(o, alone) for o in outs)
    assert torch.equal(decoded, want) and status.item() == 0 and s.status.item() == 0


@pytest.mark.parametrize("kind", ["int4", "bf16"])
def test_plain_arguments_and_others_give_the_same(kind):
    """A stream of the caller's, or a pool of a class of the caller's, takes the binding's long way."""
    class Mine(pa.Pool):
        pass
    s, _ = start(kind)
    t, _ = start(kind)
    t.pool = Mine(t.pool.k_pool, t.pool.v_pool, **(dict(k_ranges=t.ranges[0], v_ranges=t.ranges[1]) if kind == "int4" else {}))
    x = projections(len(PROMPTS), 9)
    outs = [zeros(len(PROMPTS), HQ, D, dtype=torch.bfloat16) for _ in "ab"]
    for server, out in zip((s, t), outs):
        for _ in range(3):
            server.decode(x, out)
    assert torch.equal(*outs)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    rows = ints([5, 40, 0, 12, 7])
    again = torch.empty_like(outs[0])
    q = projections(len(PROMPTS), 11)[:, :HQ].contiguous()
    pa.attention(s.pool, q, s.ids, rows, s.tables, outs[0], workspace=s.ws)
    torch.cuda.synchronize()
    pa.attention(s.pool, q, s.ids, rows, s.tables, again, workspace=s.ws, stream=stream)
    stream.synchronize()
    assert torch.equal(outs[0], again)


def test_readme_serving_step():
    """README's example of a serving step, run as it stands."""
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        block = next(b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "tables_release" in b)
    n_rows, n_seqs, num_pages = sum(PROMPTS), len(PROMPTS), 100
    bf16 = dict(dtype=torch.bfloat16)
    a = dict(pa=pa, torch=torch, num_pages=num_pages, Hkv=HKV, Hq=HQ, D=D, P=PAGE, n_rows=n_rows, n_seqs=n_seqs,
             slots=torch.arange(n_seqs, dtype=torch.int32, device="cuda"), lengths=zeros(n_seqs), new_tokens=ints(PROMPTS),
             free_pages=torch.arange(num_pages, dtype=torch.int32, device="cuda"), free_count=ints([num_pages]),
             block_tables=torch.full((n_seqs, BLOCKS), -1, dtype=torch.int32, device="cuda"), row_starts=zeros(n_seqs + 1),
             page_starts=zeros(n_seqs + 1), row_seqs=zeros(n_rows), row_positions=zeros(n_rows), qkv=projections(n_rows, 2),
             q_out=zeros(n_rows, HQ, D, **bf16), k_rows=zeros(n_rows, HKV, D, **bf16), v_rows=zeros(n_rows, HKV, D, **bf16),
             out=zeros(n_rows, HQ, D, **bf16))
    exec(block, a)
    at = a["row_starts"].tolist()
    for x, y in zip(at, at[1:]):
        want, size, _, big = R.causal(a["q_out"][x:y], a["k_rows"][x:y], a["v_rows"][x:y], R.scale_of(D))
        assert bool(((a["out"][x:y].double() - want).abs() <= R.causal_bound(want, size, D, y - x, big)).all())
    # the keys that were read back lie within a step and a half of what was rotated (half a step, and the range's f16 roundings),
    # and a rounding to bf16
    f, m = a["rope"].frequencies()
    want, _ = R.rotate(a["qkv"][:, HQ:HQ + HKV], a["row_positions"], f, m, D, False)
    step = (want.amax(dim=2, keepdim=True) - want.amin(dim=2, keepdim=True)) / 15
    assert bool(((a["k_rows"].double() - want).abs() <= 1.5 * step + want.abs() * 2.0 ** -7).all())
    assert a["free_count"].item() == num_pages and (a["block_tables"] == -1).all()
    assert sorted(a["free_pages"].tolist()) == list(range(num_pages))
