"""GPU tests of attention at the ends of FP32's range: scores that overflow or
come near it, and values that are not finite in parts of little weight."""
import numpy as np
import pytest

import attention_reference as ref
from gpu_helpers import note
from test_attention_decode_gpu import call as decode_call
from test_attention_decode_gpu import make as decode_make
from test_attention_prompt_gpu import call, check, dev, make, starts

pytestmark = pytest.mark.gpu

# Sequence, Hq, Hkv, D, kv: 16-row blocks; tiles; tiles with the keys in parts.
FORMS = [([100], 2, 1, 64, "f32"), ([100], 2, 1, 64, "f16"), ([1100], 12, 12, 64, "f32"), ([1500], 12, 12, 64, "f32"),
         ([110, 120, 100, 110], 32, 8, 128, "f16"), ([1600], 12, 12, 64, "f16")]


def name(form):
    return f"{len(form[0])}x{form[0][0]}h{form[1]}-{form[2]}d{form[3]}{form[4]}"


@pytest.mark.parametrize("form", FORMS, ids=name)
def test_a_score_that_overflows(form):
    """An infinite score makes the rows that see it NaN, as infinity minus
    infinity does, also where it lies in a tile that a row sees all of."""
    lens, Hq, Hkv, D, kv = form
    note(f"overflowing score {name(form)}")
    q, k, v = make(61, lens, lens, Hq, Hkv, D, kv)
    cu = starts(lens)
    want, bound, _ = ref.prompt(q[:, :1], k[:, :1], v[:, :1], cu, cu)
    big = np.float32(3e38 if kv == "f32" else 6e4)
    k[5, 0] = big
    q[5:cu[1]] = 10 if kv == "f32" else np.float32(1e36)
    got = call(dev(q), dev(k), dev(v), cu, cu)
    assert np.isnan(got[5:cu[1], 0]).all()
    check(got[:5, :1], want[:5], bound[:5], "rows before it")
    if len(lens) > 1:
        check(got[cu[1]:, :1], want[cu[1]:], bound[cu[1]:], "other sequences")


@pytest.mark.parametrize("form", [f for f in FORMS if f[4] == "f32"], ids=name)
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_near_the_largest_finite_value(form, sign):
    """Finite scores whose powers of two are beyond FP32: one key far above the
    others (sign 1), or all of them near the lowest finite value."""
    lens, Hq, Hkv, D, kv = form
    note(f"scores near the largest {sign} {name(form)}")
    q, k, v = make(62, lens, lens, Hq, Hkv, D, kv)
    cu = starts(lens)
    q[:] = 0
    q[:, :, 3] = 1e19
    k[:, :, 3] = -3.2e19 if sign < 0 else np.linspace(-1, 1, lens[0], dtype=np.float32)[:, None]
    k[7, :, 3] = -2.6e19 if sign < 0 else 3.2e19
    got = call(dev(q), dev(k), dev(v), cu, cu, scale=1.0)[7:, 0]
    assert (np.abs(got - v[7, 0]) <= 2.0 ** -23 * np.abs(v[7, 0])).all()


@pytest.mark.parametrize("sq,sk", [(2e-38, 2e37), (1e-39, 1e38), (1e37, 2e-38)])
def test_products_of_the_smallest_and_largest(sq, sk):
    """Rows near FP32's smallest normal value (and below) against keys near its largest."""
    note(f"smallest and largest {sq} {sk}")
    q, k, v = make(64, [1100], [1100], 12, 12, 64, "f32")
    k = np.clip(k, -3, 3)
    q, k = q * np.float32(sq), k * np.float32(sk)
    cu = starts([1100])
    got = call(dev(q), dev(k), dev(v), cu, cu)
    want, bound, _ = ref.prompt(q[:, 4:5], k[:, 4:5], v[:, 4:5], cu, cu)
    check(got[:, 4:5], want, bound)


@pytest.mark.parametrize("bad", [np.nan, np.inf])
@pytest.mark.parametrize("kv", ["f32", "f16"])
def test_values_in_parts_of_little_weight(kv, bad):
    """A value that is not finite among keys whose weights underflow beside
    another part's: 0 times it is NaN."""
    note(f"parts of little weight {bad} {kv}")
    q, k, v, table, lens = decode_make(63, [2000, 1990], 0, 16, 1, 1, 64, kv)
    want, bound = ref.decode(q, k, v, table, lens)
    q[:] = np.abs(q)
    for b in range(2):
        for j in range(100, 120):
            k[table[b, j], 0, 3] = 40
    v[table[0, 1], 0, 2, 5] = bad
    want, bound = ref.decode(q, k, v, table, lens)
    got = decode_call(dev(q), dev(k), dev(v), table, lens)
    keep = np.arange(64) != 5
    assert not np.isfinite(got[0, 0, 5])
    check(got[0, 0, keep], want[0, 0, keep], bound[0, 0, keep], "beside it")
    check(got[1], want[1], bound[1], "the other sequence")
