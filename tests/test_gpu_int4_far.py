"""Queries over a 4-bit pool of any finite size: scores are the formula's wherever they are finite, and a row whose
scores are all far below zero still has a softmax."""
import pytest
import torch

import paged_kv_continuous_pa_gb300 as pa
import serving_ref as R
import test_gpu_int4 as T

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("q_dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("exponent", [110, 117, 119, 120, 126, -100, -110])
def test_large_and_small_queries(q_dtype, d, exponent):
    """The softmax scale takes back what the queries are larger by, so the results are those of queries of size 1, for
    bf16 as exactly: the formula's bound holds for them."""
    c = T.Cache4([1, 17, 300, 4200], hkv=2, d=d, seed=exponent + 200)
    # sizes up to 3.9: below 2^(exponent + 2), finite
    q = T.queries(4, 8, d, torch.float32, seed=d).clamp(-3.9, 3.9).bfloat16().double()
    q = (q * 2.0 ** exponent).to(q_dtype)
    assert torch.isfinite(q).all()
    T.check(c, q, c.slots, [n - 1 for n in c.lengths], softmax_scale=R.scale_of(d) * 2.0 ** -exponent)


@pytest.mark.parametrize("q_dtype", DTYPES)
def test_queries_of_one_sign(q_dtype):
    """Elements whose sum is beyond the largest number, where no score is."""
    c = T.Cache4([40, 700], hkv=2, d=128, page=32, seed=3)
    q = (T.queries(2, 8, 128, torch.float32).abs().clamp(max=1.9) + 2.0).bfloat16().double()
    assert float(q.sum(dim=2).min()) > 2.0 ** 8
    q = (q * 2.0 ** 125).to(q_dtype)
    assert torch.isfinite(q).all() and not torch.isfinite(q.float().sum(dim=2)).any()
    T.check(c, q, c.slots, [39, 699], softmax_scale=R.scale_of(128) * 2.0 ** -127)


@pytest.mark.parametrize("q_dtype", DTYPES)
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_far_from_zero(q_dtype, sign):
    """All scores of a row near 2^124 or -2^124: tokens of one key each share the weight, others get none, whatever
    the others' distance.  Keys are one value each (step 0), so their scores are exactly alike."""
    c = T.Cache4([1, 40, 4200], hkv=2, d=64, page=16, seed=5)
    c.ranges[0][..., 0] = 0.0
    c.ranges[0][..., 1] = 1.0  # a score is the sum of the query's elements
    best = {c.slots[0]: [0], c.slots[1]: [3, 37], c.slots[2]: [11, 700, 4199]}
    for slot, tokens in best.items():
        for t in tokens:
            c.ranges[0][int(c.tables[slot, t // 16]), :, t % 16, 1] = 2.0 if sign > 0 else 0.5
    q = torch.full((3, 8, 64), sign * 2.0 ** 120, device="cuda", dtype=q_dtype)
    out, status = T.attend(c, q, c.slots, [0, 39, 4199])
    assert status == 0
    for r, slot in enumerate(c.slots):
        v = c.cached(1, slot, (1, 40, 4200)[r])[0][:, best[slot]]  # [Hkv, best, D]
        want = v.mean(dim=1).repeat_interleave(4, 0)
        # equal weights, exact but for their f16 products with the step (2^-11 for bf16 rows, 2^-22), and the output's rounding
        size = v.abs().amax(dim=(1, 2), keepdim=True).squeeze(1).repeat_interleave(4, 0) * 16
        rel = 2.0 ** -11 if q_dtype == torch.bfloat16 else 2.0 ** -21
        assert ((out[r].double() - want).abs() <= rel * size + R.HALF_STEP[q_dtype] * (want.abs() + rel * size)).all()
