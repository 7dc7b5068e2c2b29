"""Infinite values in every unit of pa_prompt_attention's work at once: units of one and two key blocks in turn, head
groups whose two tiles are ranges of one head and pairs of heads."""
import pytest
import torch

import paged_kv_continuous_pa_gb300 as pa
import test_gpu_prompt as P

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d", [(3, 3, 64), (3, 1, 128), (4, 2, 64)])
def test_infinite_values_in_every_unit(hq, hkv, d):
    lengths = ([200] + [50, 128, 1, 90, 60, 3] * 2 + [256, 20]) * 30  # 450 sequences, more units than CTAs
    q, k, v, starts = P.make(lengths, hq, hkv, d, seed=hq * d, packed=True)
    at = starts.tolist()
    clean, status = P.run(q, k, v, starts)
    assert status == 0 and torch.isfinite(clean.float()).all()
    expect = clean.float()
    v = v.clone()
    for i, (a, b) in enumerate(zip(at, at[1:])):
        # one value of each kind, in the sequence's last token and somewhere before it
        for column, key, value in ((3, b - 1, float("inf")), (7, a + (i * 13) % (b - a), float("nan"))):
            v[key, :, column] = value
            expect[key:b, :, column] = value
    for _ in range(20):
        out, status = P.run(q, k, v, starts)
        assert status == 0
        assert torch.equal(torch.isnan(out), torch.isnan(expect))
        fine = ~torch.isnan(expect)
        assert torch.equal(out.float()[fine], expect[fine])
