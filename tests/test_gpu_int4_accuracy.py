"""Accuracy of attention over a 4-bit pool as the norm of the error against the norm of the result: f32 rows keep what FP32
sums keep, and queries with a common offset cost bf16 rows nothing beside their output's rounding."""
import pytest
import torch

import paged_kv_continuous_pa_gb300 as pa
import serving_ref as R
import test_gpu_int4 as T

pytestmark = pytest.mark.gpu


def error(c, q, lengths, softmax_scale=None):
    """(error, error of the exact result rounded to the type), of the result's norm."""
    scale = softmax_scale or R.scale_of(c.d)
    out, status = T.attend(c, q, c.slots, [n - 1 for n in lengths], softmax_scale=scale)
    assert status == 0
    want = torch.stack([R.attend4(q[i], c.cached(0, s, n)[0], c.cached(1, s, n)[0], scale)[0]
                        for i, (s, n) in enumerate(zip(c.slots, lengths))])
    rounded = want.to(q.dtype).double() - want
    return float((out.double() - want).norm() / want.norm()), float(rounded.norm() / want.norm())


# Weights of f32 rows.  A score in the log2 domain is of size 1.5 (queries and values of size 1, scale 1 / sqrt(D)); its
# sums over centred codes go through 16 truncations of 2^-23 of partial sums below 4: each is off by a number spread over one
# unit, 0.29 units beside its mean, which a softmax divides out, so 4 x 0.29 x 2 x 2^-23 x ln 2 = 1.6 x 2^-23.  ex2 is off by
# 2^-22 at most, the weight's second part by 2^-23: weights by 2^-21.5 in all, independent of one another, and so the
# result against its norm.  The sums of weights times centred values are of the result's own size, 16 tokens at a time: a
# unit of 2^-23 each, as the sums of low + 8 step, which are up to sqrt(length) / 8 times as large as a result of
# length terms: 2^-22 at 4200.  2^-21 in all, and twice that allowed.
F32_NORM = 2.0 ** -20


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_f32_rows_of_every_group(G, d):
    lengths = [33, 100, 700, 701, 53, 350, 1000, 64]
    c = T.Cache4(lengths, hkv=4, d=d, page=32, seed=G)
    err, _ = error(c, T.queries(8, 4 * G, d, torch.float32, seed=G), lengths)
    assert err <= F32_NORM, err


@pytest.mark.parametrize("d", [64, 128])
def test_f32_rows_in_splits(d):
    lengths = [4097, 4200, 6000, 5001]
    c = T.Cache4(lengths, hkv=2, d=d, page=64, seed=d)
    q = T.queries(4, 8, d, torch.float32, seed=d)
    err, _ = error(c, q, lengths)
    assert err <= F32_NORM, err
    old = pa.get_split_tokens()
    pa.set_split_tokens(64)
    try:
        err, _ = error(c, q, lengths)
    finally:
        pa.set_split_tokens(old)
    assert err <= F32_NORM, err


@pytest.mark.parametrize("offset", [0.0, 1.0, 4.0, 16.0, 64.0, 256.0])
@pytest.mark.parametrize("d,length", [(64, 53), (128, 700), (128, 4096)])
def test_bf16_rows_with_an_offset(d, length, offset):
    """step (q . c) and low sum(q) are large and opposite then.  Scores may be cut off at 2^-18 of their largest product (in
    subnormal numbers), 15 step (1 + offset) scale: 8 products' sums of it are 2^-11 (1 + offset) step scale, which with
    step < 0.4 and a scale of 1 / (sqrt(D) (1 + offset)) is below 2^-14; weights in f16 2^-12.  Beside the output's rounding,
    2^-9.3 of the norm, that is a fifth of it at most, and errors of other causes add up as squares: 1.05."""
    c = T.Cache4([length] * 8, hkv=4, d=d, page=32, seed=length)
    q = (T.queries(8, 16, d, torch.float32, seed=d) + offset).bfloat16()
    err, rounding = error(c, q, [length] * 8, R.scale_of(d) / (1 + offset))
    assert err <= 1.05 * rounding, (err, rounding)
