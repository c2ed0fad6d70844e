"""Scales of an 8-bit cache that the append refuses, on the CPU, with pointers
that are never read."""
import pytest

from row_reduction_norm_gb300 import _native as N
from test_rope_host import app, paged


# the inverse of the first is not finite in fp32; next to the limits 2^-100 and 2^100
@pytest.mark.parametrize("scale", [1e-39, 2.0 ** -149, 2.0 ** -101, 0.999 * 2.0 ** -100, 1.001 * 2.0 ** 100, 2.0 ** 127])
@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
def test_scales_out_of_range_are_refused(which, scale):
    assert app(kv=paged(cache_dtype=N.RMSNORM_E4M3, **{which: scale})) == N.RMSNORM_EINVAL


@pytest.mark.parametrize("scale", [2.0 ** -100, 0.05, 1.0, 2.0 ** 100])
def test_scales_in_range_are_taken(scale):
    """As far as an empty batch shows it; caches of the I/O type have no scale."""
    kv = paged(cache_dtype=N.RMSNORM_E4M3, k_scale=scale, v_scale=scale)
    assert app(x=None, qo=None, tokens=0, kv=kv) == N.RMSNORM_OK
    assert app(x=None, qo=None, tokens=0, kv=paged(k_scale=0.0, v_scale=1e-39)) == N.RMSNORM_OK
