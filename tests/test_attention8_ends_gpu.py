"""GPU tests of attention over an 8-bit cache beyond FP32's range, as the header has it."""
import numpy as np
import pytest

import compensated_fp32_projection_amd as cf
from gpu_helpers import note
from test_attention8_gpu import expected, problem
from test_cache8_gpu import cache_of, dev, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("n", [3, 70, 3000])
def test_scores_beyond_the_range(n, kind):
    """Row 0: every score -infinite; row 1: one +infinite; row 2: one -infinite, which counts for nothing; row 3 ordinary."""
    rng = np.random.default_rng(n)
    q, arrays, table, lens = problem(rng, [n], 4, 4, 64, 16, 1, kind)
    arrays[0][:] = np.where(arrays[0].view(np.int8) == 0, 1, arrays[0] & 0x3F | 1)  # codes of at least 1 (floats: 2^-9)
    q = np.abs(q) + np.float32(0.1)
    keys = arrays[1].transpose(0, 2, 1)  # [pages, tokens, heads], of the table's pages
    some = (table[0, n // 2 // 16], n // 2 % 16)
    keys[..., 0] = 2.0 ** 100
    q[0, 0] *= np.float32(-2.0 ** 60)
    keys[some + (1,)], keys[some + (2,)] = 2.0 ** 100, 2.0 ** 100
    q[0, 1] *= np.float32(2.0 ** 60)
    q[0, 2] *= np.float32(-2.0 ** 60)
    keys[..., 1:3] = np.where(keys[..., 1:3] < 2.0 ** 99, keys[..., 1:3] * 2.0 ** -60, keys[..., 1:3])
    arrays[1] = np.ascontiguousarray(keys.transpose(0, 2, 1)).astype(np.float32)
    c, *_ = cache_of(arrays, kind)
    note(f"decode8 scores beyond {n} {kind}")
    got, = host(cf.attention8_decode(dev(q), c, dev(table), dev(lens)))
    want, bound = expected(q, arrays, kind, 1, table, lens)
    assert (got[0, 0] == 0).all() and np.isnan(got[0, 1]).all()
    assert (np.abs(got[0, 2:] - want[0, 2:]) <= bound[0, 2:]).all()


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_sums_beyond_the_range(kind):
    """Values of 2^127 in one head of two: its rows are not finite, the other head's are as they are."""
    rng = np.random.default_rng(1)
    q, arrays, table, lens = problem(rng, [100], 2, 2, 64, 16, 16, kind)
    arrays[2][:, 0] = 64 if kind == "i8" else 0x68  # 64
    arrays[3][:, 0] = 2.0 ** 121
    c, *_ = cache_of(arrays, kind)
    note(f"decode8 sums beyond {kind}")
    got, = host(cf.attention8_decode(dev(q * np.float32(1e-3)), c, dev(table), dev(lens)))
    want, bound = expected(q * np.float32(1e-3), arrays, kind, 16, table, lens)
    assert not np.isfinite(got[0, 0]).any()
    assert (np.abs(got[0, 1] - want[0, 1]) <= bound[0, 1]).all()
