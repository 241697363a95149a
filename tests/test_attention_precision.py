"""What the precision measure of attention_precision.py notices, on the CPU."""
import numpy as np
import pytest

import attention_precision as ap


def one_part(x):
    return x.astype(np.float16).astype(np.float32)


def two_parts(x):
    hi = one_part(x)
    return hi + one_part(x - hi)


@pytest.mark.parametrize("n,D,shared", [(1100, 64, False), (300, 128, False), (6000, 64, True)])
def test_the_measure_tells_one_part_from_two(n, D, shared):
    """An operand (the weights among them) in one FP16 part is far outside, all of them in two inside."""
    rng = np.random.default_rng(n + D)
    rows = 40 if shared else n
    q = rng.standard_normal((rows, D), dtype=np.float32) * 1.5
    k = rng.standard_normal((n, D), dtype=np.float32)
    v = rng.standard_normal((n, D), dtype=np.float32)
    limits, scale = np.full(rows, n) if shared else np.arange(1, n + 1), D ** -0.5
    want, norm = ap.exact(q, k, v, limits, scale)
    base = ap.rms((ap.plain(q, k, v, limits, scale) - want) / norm)
    for name in "qkvw":
        cut = ap.plain(q, k, v, limits, scale, lambda at, x: one_part(x) if at == name else x)
        assert ap.rms((cut - want) / norm) > 8 * ap.RATIO * base, name
    both = ap.plain(q, k, v, limits, scale, lambda at, x: two_parts(x * np.float32(2048)) / np.float32(2048))
    assert ap.rms((both - want) / norm) <= ap.RATIO * base
