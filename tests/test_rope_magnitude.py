"""The factor on rotated pairs: what a ramp takes where none is given, and numbers that FP32 does not hold."""
import math

import pytest

import paged_kv_continuous_pa_gb300 as pa
from paged_kv_continuous_pa_gb300 import build as pa_build


@pytest.fixture(scope="module", autouse=True)
def lib():
    pa_build.build()
    return pa.load()


def ramp(factor, **kw):
    return pa.Rope(64, scaling="ramp", factor=factor, original_positions=4096, **kw)


@pytest.mark.parametrize("factor", [1.0, 0.9, 0.5, 2.0 ** -4, 4.5e-5, 1e-5, 1e-12])
def test_ramps_that_stretch_nothing_keep_the_size(factor):
    """0.1 ln(factor) + 1 would shrink queries and keys, and from e^-10 on turn them around."""
    assert ramp(factor).frequencies()[1] == 1.0


@pytest.mark.parametrize("factor", [1.0 + 2.0 ** -40, 1.5, 8.0, 1e6])
def test_ramps_that_stretch(factor):
    assert ramp(factor).frequencies()[1] == pytest.approx(0.1 * math.log(factor) + 1.0, rel=1e-15)


def test_a_given_magnitude_stays():
    assert ramp(1e-5, magnitude=0.25).frequencies()[1] == 0.25 and ramp(8.0, magnitude=1.0).frequencies()[1] == 1.0


@pytest.mark.parametrize("magnitude", [1e39, 1e300, 1e-46, 5e-324])
def test_magnitudes_beyond_fp32_are_refused(magnitude):
    """The kernels hold it in FP32, where these are infinite or 0."""
    with pytest.raises(pa.PaError) as e:
        pa.Rope(64, magnitude=magnitude)
    assert e.value.status == pa.PA_ERR_INVALID_ARG


@pytest.mark.parametrize("magnitude", [3e38, 1e-44, 1.0])
def test_magnitudes_of_fp32(magnitude):
    assert pa.Rope(64, magnitude=magnitude).frequencies()[1] == magnitude
