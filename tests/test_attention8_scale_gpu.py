"""GPU tests of attention over an 8-bit cache with scales of the scores at the ends of FP32's range."""
import numpy as np
import pytest

import compensated_fp32_projection_amd as cf
from gpu_helpers import note
from test_attention8_gpu import check, expected, problem
from test_cache8_gpu import cache_of, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("scale,qs", [(3e38, 2.0 ** -124), (-3e38, 2.0 ** -124), (2.0 ** 121, 2.0 ** -118), (2.0 ** -140, 2.0 ** 100)])
def test_scales_at_the_ends_of_the_range(scale, qs, kind):
    """Scales near the largest finite value, or below the normal ones, with rows that bring the scores back."""
    rng = np.random.default_rng(3)
    q, arrays, table, lens = problem(rng, [200, 17], 4, 2, 64, 16, 16, kind)
    q = (q * np.float32(qs)).astype(np.float32)
    if scale == 2.0 ** -140:
        arrays[1] = (arrays[1] * np.float32(2.0 ** 40)).astype(np.float32)
    c, *_ = cache_of(arrays, kind)
    note(f"decode8 scale {scale} {kind}")
    check(cf.attention8_decode(dev(q), c, dev(table), dev(lens), scale=scale), expected(q, arrays, kind, 16, table, lens, scale))
