"""Calls from threads of the caller's own: a thread's first CUDA call, and
several threads' first calls on one pool."""
import threading

import pytest
import torch

import cache_ref as R
import paged_kv_continuous_pa_gb300 as pa

pytestmark = pytest.mark.gpu

ROWS = 40


class Step:
    """One chunk of ROWS rows, and what each call gives on the main thread."""

    def __init__(self, kv, q_dtype=torch.bfloat16):
        self.c = c = R.make_cache([900], Hkv=2, D=128, P=32, kv=kv, seed=35)
        g = torch.Generator().manual_seed(35)
        self.q = torch.randn(ROWS, 8, 128, generator=g).to(q_dtype).cuda()
        self.ids = torch.tensor(c.slots * ROWS, dtype=torch.int32, device="cuda")
        self.pos = torch.arange(900 - ROWS, 900, dtype=torch.int32, device="cuda")
        self.want = self.buffers()
        for name in self.calls():
            self.calls()[name](c.pool, self.want, None)
        torch.cuda.synchronize()

    def chunked(self, name):
        return [(0, ROWS)] if name != "rows" else []

    def buffers(self):
        c, out = self.c, {}
        for name in self.calls():
            size = (pa.mass_workspace_bytes if name == "mass" else pa.workspace_bytes)(c.pool, ROWS, 8, c.max_blocks, self.chunked(name))
            ws = torch.zeros(max(size, 1), dtype=torch.uint8, device="cuda")
            res = torch.zeros(c.num_seqs, c.Hkv, c.max_tokens, device="cuda") if name == "mass" else torch.zeros_like(self.q)
            out[name] = (res, ws)
        torch.cuda.synchronize()
        return out

    def calls(self):
        def mass(pool, to, stream):
            res, ws = to["mass"]
            pa.attention_mass(pool, self.q, self.ids, self.pos, self.c.tables, res, chunks=[(0, ROWS)], workspace=ws, stream=stream)

        def attend(name):
            def call(pool, to, stream):
                res, ws = to[name]
                pa.attention(pool, self.q, self.ids, self.pos, self.c.tables, res, chunks=self.chunked(name), workspace=ws, stream=stream)
            return call
        return {"mass": mass, "chunk": attend("chunk"), "rows": attend("rows")}

    def pool(self):
        scale = self.c.scale.view(-1).cpu().float().numpy() if self.c.kv == "e4m3" else 1.0
        return pa.Pool(self.c.k, self.c.v, scale, scale)


def in_threads(work):
    errors = []

    def guarded(f):
        try:
            f()
        except Exception as e:
            errors.append(e)
    threads = [threading.Thread(target=guarded, args=(f,)) for f in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", ["mass", "chunk", "rows"])
@pytest.mark.parametrize("fresh", [True, False])
def test_first_call_of_a_thread(kv, name, fresh):
    """The thread has no context yet, and gives a stream, so that nothing sets one up before the call."""
    s = Step(kv)
    got, stream = s.buffers(), torch.cuda.Stream()
    pool = s.pool() if fresh else s.c.pool
    in_threads([lambda: s.calls()[name](pool, got, stream)])
    assert torch.equal(got[name][0], s.want[name][0])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_first_calls_of_a_pool(kv):
    """The pool's tensor maps are encoded by whichever call comes first, whole before any call reads them."""
    s = Step(kv)
    names = ["mass", "chunk", "rows"] * 2
    for _ in range(8):
        pool, gate = s.pool(), threading.Barrier(len(names))
        got, streams = [s.buffers() for _ in names], [torch.cuda.Stream() for _ in names]

        def work(i):
            gate.wait()
            s.calls()[names[i]](pool, got[i], streams[i])
        in_threads([lambda i=i: work(i) for i in range(len(names))])
        for name, to in zip(names, got):
            assert torch.equal(to[name][0], s.want[name][0])
