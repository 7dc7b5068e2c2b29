"""Angles at positions up to the ends of int32, against integers of 200 bits: the position times f_i modulo whole turns
is that of the f_i that Rope.frequencies() gives, without an error that grows with the position."""
import pytest
import torch

import paged_kv_continuous_pa_gb300 as pa
import serving_ref as R
import test_gpu_rope as T

pytestmark = pytest.mark.gpu
PI = 314159265358979323846264338327950288419716939937510582097494459  # times 10^62
BITS = 200


def turns(f):
    """f / 2 pi as a whole number of 2^-200 turns (f: a double, a whole number over a power of two)."""
    num, den = float(f).as_integer_ratio()
    return (num << BITS) * 10 ** 62 // (2 * PI * den)


def rotate(x, positions, frequencies, magnitude, rot, interleaved):
    """serving_ref.rotate with exact angles: the fraction of a turn in 64 bits, then as a double."""
    f = [turns(v) for v in frequencies]
    angle = torch.tensor([[float((p * v) % (1 << BITS) >> (BITS - 64)) * 2.0 ** -64 for v in f] for p in positions.tolist()],
                         dtype=torch.float64, device=x.device).unsqueeze(1) * (2 * torch.pi)
    x = x.double()
    c, s = angle.cos() * magnitude, angle.sin() * magnitude
    out, size = x.clone(), torch.zeros_like(x)
    i = torch.arange(rot // 2, device=x.device)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    a, b = x[:, :, ia], x[:, :, ib]
    out[:, :, ia], out[:, :, ib] = a * c - b * s, a * s + b * c
    size[:, :, ia] = size[:, :, ib] = (a.abs() + b.abs()) * magnitude
    return out, size


@pytest.mark.parametrize("kw", [dict(), dict(base=1.5), dict(base=500000.0, scaling="bands", factor=8.0, original_positions=8192),
                                dict(scaling="linear", factor=0.5), dict(scaling="linear", factor=0.01),
                                dict(scaling="linear", factor=1e-12)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_positions(kw, layout):
    """serving_ref.rotate_bound, whose terms count no error of the angle itself but its rounding to FP32."""
    g = torch.Generator().manual_seed(3)
    positions = torch.randint(-2 ** 31, 2 ** 31, (3000,), generator=g).to(torch.int32)
    positions[:4] = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 31 - 2, 1])
    x = T.normal((3000, 1, 64), torch.float32, 4)
    rope = pa.Rope(64, layout=layout, **kw)
    out = torch.empty_like(x)
    pa.rope_rows(rope, x, positions.cuda(), out)
    f, m = rope.frequencies()
    want, size = rotate(x, positions, f, m, 64, layout == "interleaved")
    err, bound = (out.double() - want).abs(), R.rotate_bound(size, want, torch.float32)
    assert (err <= bound).all(), f"{float((err / bound).max()):.3g} of the bound"
