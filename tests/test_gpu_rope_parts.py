"""rope_rows on a part of a packed projection: in place, from one stride to another, one row, and nothing beside it touched."""
import pytest
import torch

import paged_kv_continuous_pa_gb300 as pa
import test_gpu_rope as T

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("layout,d,rot", [("half", 128, 128), ("half", 64, 20), ("interleaved", 64, 32)])
@pytest.mark.parametrize("n", [1, 9, 1300])
@pytest.mark.parametrize("first,heads", [(0, 6), (6, 2), (8, 2)])
def test_parts(dtype, layout, d, rot, n, first, heads):
    qkv = T.normal((n, 10, d), dtype, n + d)
    positions = torch.randint(0, 200000, (n,), dtype=torch.int32, generator=torch.Generator().manual_seed(n)).cuda()
    rope = pa.Rope(rot, layout=layout, magnitude=1.25)
    part = lambda x: x[:, first:first + heads]
    for inverse in (False, True):
        want = torch.empty(n, heads, d, dtype=dtype, device="cuda")
        pa.rope_rows(rope, part(qkv), positions, want, inverse=inverse)
        T.assert_rotated(want, part(qkv), positions, rope, rot, layout == "interleaved", inverse)
        # in place, its neighbours as they were
        same = qkv.clone()
        pa.rope_rows(rope, part(same), positions, inverse=inverse)
        assert torch.equal(part(same), want)
        # into a part of another projection, of another stride
        wide = torch.full((n, 13, d), 7.0, dtype=dtype, device="cuda")
        pa.rope_rows(rope, part(qkv), positions, wide[:, 11 - heads:11], inverse=inverse)
        assert torch.equal(wide[:, 11 - heads:11], want)
        # from contiguous rows into a part
        wide2 = torch.full((n, 13, d), 7.0, dtype=dtype, device="cuda")
        pa.rope_rows(rope, part(qkv).contiguous(), positions, wide2[:, 11 - heads:11], inverse=inverse)
        assert torch.equal(wide2, wide)
        keep = torch.ones(10, dtype=torch.bool)
        keep[first:first + heads] = False
        assert torch.equal(same[:, keep], qkv[:, keep])
        assert (wide[:, :11 - heads] == 7.0).all() and (wide[:, 11:] == 7.0).all()
