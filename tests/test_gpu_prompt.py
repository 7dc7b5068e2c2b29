"""pa_prompt_attention against a 64-bit reference: lengths, head groups, packed rows,
poisoned strangers, infinite values, refusals on the device, graphs."""
import pytest
import torch

import paged_kv_continuous_pa_gb300 as pa
import serving_ref as R

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def rows(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(BF16).cuda()


def make(lengths, hq, hkv, d, seed=0, packed=False, pad=0, gap=0, scale=1.0):
    n = gap + sum(lengths) + pad
    qkv = rows((n, hq + 2 * hkv, d), seed, scale)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    starts = torch.tensor([gap + sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")
    return q, k, v, starts


def run(q, k, v, starts, out=None, lse=None, **kw):
    n, hq, d = q.shape
    out = torch.full((n, hq, d), 7.0, dtype=BF16, device="cuda") if out is None else out
    size = pa.prompt_workspace_bytes(n, starts.numel() - 1, hq, k.shape[1], d)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda").fill_(0xA5)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.prompt_attention(q, k, v, starts, out, lse=lse, workspace=ws, status=status, **kw)
    torch.cuda.synchronize()
    return out, int(status.item())


def check(q, k, v, starts, softmax_scale=None, with_lse=False):
    n, hq, d = q.shape
    scale = softmax_scale or R.scale_of(d)
    lse = torch.full((n, hq), 7.0, device="cuda") if with_lse else None
    out, status = run(q, k, v, starts, lse=lse, softmax_scale=softmax_scale or 0.0)
    assert status == 0
    at = starts.tolist()
    untouched = torch.ones(n, dtype=torch.bool, device="cuda")
    for a, b in zip(at[:-1], at[1:]):
        if a == b:
            continue
        want, size, total, big = R.causal(q[a:b], k[a:b], v[a:b], scale)
        bound = R.causal_bound(want, size, d, b - a, big)
        err = (out[a:b].double() - want).abs()
        assert (err <= bound).all(), f"rows {a}..{b}: {float((err / bound).max()):.3g} of the bound"
        if with_lse:
            assert ((lse[a:b].double() - total).abs() <= 2 * R.score_error(d, big) + 2.0 ** -20 + (b - a) * 2.0 ** -23
                    + total.abs() * 2.0 ** -22).all()
        untouched[a:b] = False
    assert (out[untouched] == 7.0).all()
    if with_lse:
        assert (lse[untouched] == 7.0).all()
    return out


@pytest.mark.parametrize("length", [1, 2, 31, 127, 128, 129, 255, 256, 257, 383, 385, 700])
@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 128), (3, 3, 128), (4, 2, 64), (5, 1, 64)])
def test_lengths(length, hq, hkv, d):
    check(*make([length], hq, hkv, d, seed=length), with_lse=True)


@pytest.mark.parametrize("group", [1, 2, 3, 4, 7, 8, 16])
@pytest.mark.parametrize("packed", [False, True])
def test_groups(group, packed):
    check(*make([5, 300, 129], 2 * group, 2, 128, seed=group, packed=packed, pad=3))


@pytest.mark.parametrize("hq,hkv", [(4, 2), (3, 1)])
def test_ragged(hq, hkv):
    """Many short sequences, empty ones among them, rows before the first and behind the last."""
    lengths = [(i * 37) % 200 for i in range(90)] + [0, 0, 1, 0]
    check(*make(lengths, hq, hkv, 64, seed=1, packed=True, pad=50, gap=11), with_lse=True)


@pytest.mark.parametrize("length", [2048, 4133])
@pytest.mark.parametrize("hq,hkv,d", [(2, 1, 128), (1, 1, 64)])
def test_long(length, hq, hkv, d):
    check(*make([length, 60], hq, hkv, d, seed=length), with_lse=True)


def test_more_sequences_than_threads():
    check(*make([3] * 1500, 2, 2, 64, seed=4))


@pytest.mark.parametrize("softmax_scale", [0.01, 1.5])
@pytest.mark.parametrize("hq", [2, 1])
def test_scales(softmax_scale, hq):
    check(*make([500], hq, 1, 128, seed=8), softmax_scale=softmax_scale)


@pytest.mark.parametrize("hq", [2, 1])
def test_growing_scores(hq):
    """Scores that rise along the keys move the reference many times; ones that fall, never."""
    for way in (1.0, -1.0):
        q, k, v, starts = make([900], hq, 1, 64, seed=9)
        ramp = torch.linspace(-1, 1, 900, device="cuda").view(-1, 1, 1) * way
        q = (q.float() * 0.1 + 2.0).to(BF16)
        k = (k.float() * 0.1 + 3.0 * ramp).to(BF16)
        check(q, k, v, starts, with_lse=True)


@pytest.mark.parametrize("hq,hkv", [(4, 2), (3, 1)])
@pytest.mark.parametrize("poison", [float("nan"), float("inf"), float("-inf")])
def test_strangers(hq, hkv, poison):
    """What other sequences, later tokens and rows outside every sequence hold has no influence."""
    lengths = [100, 140, 129]
    q, k, v, starts = make(lengths, hq, hkv, 64, seed=3, pad=140, gap=5)
    plain, status = run(q, k, v, starts)
    assert status == 0
    a, b = 105, 245  # the second sequence
    for x in (q, k, v):
        keep = x[a:b].clone()
        x.fill_(poison)
        x[a:b] = keep
    out, status = run(q, k, v, starts)
    assert status == 0
    assert torch.equal(out[a:b], plain[a:b])
    # later tokens of the sequence itself: rows before them stay as they were
    for cut in (139, 128, 127, 77, 1):
        k2, v2 = k.clone(), v.clone()
        k2[a + cut:b] = poison
        v2[a + cut:b] = poison
        out, status = run(q, k2, v2, starts)
        assert torch.equal(out[a:a + cut], plain[a:a + cut])


@pytest.mark.parametrize("hq", [2, 1])
def test_infinite_values(hq):
    """A row that attends to an infinite value gets it, one that attends to both or to NaN gets NaN."""
    q, k, v, starts = make([400], hq, 1, 64, seed=5)
    clean, _ = run(q, k, v, starts)
    v[390, 0, 3] = float("inf")
    v[395, 0, 3] = float("-inf")
    v[270, 0, 7] = float("nan")
    out, status = run(q, k, v, starts)
    assert status == 0
    expect = clean.clone().float()
    expect[390:395, :, 3] = float("inf")
    expect[395:, :, 3] = float("nan")
    expect[270:, :, 7] = float("nan")
    assert torch.equal(torch.isnan(out), torch.isnan(expect))
    fine = ~torch.isnan(expect)
    assert torch.equal(out.float()[fine], expect[fine])


def test_alone_and_in_a_batch():
    """A sequence's bits are its own, in any company and place; calls repeat themselves."""
    lengths = [260, 1, 700, 128]
    q, k, v, starts = make(lengths, 4, 2, 128, seed=6)
    out, _ = run(q, k, v, starts)
    again, _ = run(q, k, v, starts)
    assert torch.equal(out, again)
    at = starts.tolist()
    for a, b in zip(at[:-1], at[1:]):
        alone, _ = run(q[a:b].contiguous(), k[a:b].contiguous(), v[a:b].contiguous(),
                       torch.tensor([0, b - a], dtype=torch.int32, device="cuda"))
        assert torch.equal(alone, out[a:b])


@pytest.mark.parametrize("starts", [[0, 10, 5, 20], [-1, 10], [0, 21], [3, 30, 20]])
def test_bad_starts(starts):
    q, k, v, _ = make([20], 2, 1, 64)
    out, status = run(q, k, v, torch.tensor(starts, dtype=torch.int32, device="cuda"))
    assert status == pa.PA_ERR_OUT_OF_RANGE and (out == 7.0).all()


def test_wait_that_runs_out():
    q, k, v, starts = make([200], 2, 1, 64)
    pa.set_wait_limit(2000)
    pa.debug_stall_waits(True)
    try:
        _, status = run(q, k, v, starts)
    finally:
        pa.debug_stall_waits(False)
        pa.set_wait_limit(0)
    assert status == pa.PA_ERR_TIMEOUT
    check(q, k, v, starts)


def test_graph_and_stream():
    """Captured on another stream; replays follow new inputs and new lengths."""
    q, k, v, starts = make([300, 200], 4, 2, 64, seed=1, pad=40)
    out = torch.zeros(q.shape, dtype=BF16, device="cuda")
    ws = torch.empty(pa.prompt_workspace_bytes(540, 2, 4, 2, 64), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        pa.prompt_attention(q, k, v, starts, out, workspace=ws)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pa.prompt_attention(q, k, v, starts, out, workspace=ws)
    for lengths, seed in (([300, 200], 2), ([17, 523], 3)):
        q2, k2, v2, starts2 = make(lengths, 4, 2, 64, seed=seed, pad=540 - sum(lengths))
        for a, b in ((q, q2), (k, k2), (v, v2), (starts, starts2)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        want, _ = run(q2, k2, v2, starts2)
        assert torch.equal(out[:sum(lengths)], want[:sum(lengths)])


@pytest.mark.parametrize("seqs", [1, 31, 32, 33, 40])
def test_few_units_and_a_list(seqs):
    """A CTA for each unit finds its own among up to 32 sequences; beyond, they come from a list."""
    lengths = [(37 * i) % 61 for i in range(seqs)]
    check(*make(lengths, 4, 2, 64, seed=seqs), with_lse=True)


def test_groups_of_sequences():
    """Keys and values of more than one share of L2: sequences of all lengths, equal and empty ones among them."""
    lengths = [0, 700, 1, 300, 300, 300, 129, 0, 2100, 5, 64, 300, 900, 1500, 128, 0]
    check(*make(lengths, 16, 16, 128), with_lse=True)


def test_as_many_groups_as_there_are():
    """65536 rows in groups of 1024, with empty sequences behind the last row of the last group."""
    lengths = [0, 0] + [128] * 510 + [256] + [0] * 3
    g = torch.Generator(device="cuda").manual_seed(5)
    q, k, v = (torch.randn(sum(lengths), 32, 128, generator=g, device="cuda", dtype=BF16) for _ in "qkv")
    starts = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")
    out, status = run(q, k, v, starts)
    assert status == 0
    half = torch.cat([starts[:257], starts[256:257]])
    n = int(half[-1])
    part, status = run(q[:n], k[:n], v[:n], half)
    assert status == 0 and torch.equal(part, out[:n])
    back = starts[257:] - starts[257]
    m = int(starts[257])
    part, status = run(q[m:].contiguous(), k[m:].contiguous(), v[m:].contiguous(), back)
    assert status == 0 and torch.equal(part, out[m:])
    for a, b in ((0, 128), (65280, 65536), (30080, 30208)):
        want, size, _, big = R.causal(q[a:b], k[a:b], v[a:b], R.scale_of(128))
        assert bool(((out[a:b].double() - want).abs() <= R.causal_bound(want, size, 128, b - a, big)).all())


@pytest.mark.parametrize("bad", [(20, -1), (20, 10 ** 9), (39, 4000)])
def test_bad_starts_of_a_list(bad):
    q, k, v, starts = make([64] * 40, 2, 1, 64)
    starts = starts.clone()
    starts[bad[0]] = bad[1]
    out, status = run(q, k, v, starts)
    assert status == pa.PA_ERR_OUT_OF_RANGE and (out == 7.0).all()


def test_a_list_that_is_waited_for_in_vain():
    q, k, v, starts = make([200] * 40, 2, 1, 64)
    want, status = run(q, k, v, starts)
    assert status == 0
    pa.set_wait_limit(2000)
    pa.debug_stall_waits(True)
    try:
        assert run(q, k, v, starts)[1] == pa.PA_ERR_TIMEOUT
    finally:
        pa.debug_stall_waits(False)
        pa.set_wait_limit(0)
    out, status = run(q, k, v, starts)
    assert status == 0 and torch.equal(out, want)
