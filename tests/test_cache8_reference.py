"""The 8-bit cache's oracle against what torch's own conversions say, and against its bounds; no GPU."""
import numpy as np
import pytest
import torch

import cache8_reference as ref


def test_float_codes_are_torchs():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    finite = np.isfinite(want)
    assert finite.sum() == 254 and np.array_equal(ref.values(codes, "e4m3")[finite], want[finite])
    assert list(ref.values(codes, "e4m3")[~finite]) == [480.0, -480.0]


def test_rounding_to_floats_is_torchs():
    g = np.random.default_rng(0)
    y = np.concatenate([g.uniform(-448, 448, 20000), g.standard_normal(20000) * 0.01,
                        [0.0, -0.0, 2.0 ** -10, 3 * 2.0 ** -10, 448.0, -448.0, 17.0, 19.0, 2.0 ** -6, 2.0 ** -7]])
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.nearest(y, "e4m3"), want)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_values_stay_within_their_steps(kind):
    """Tokens written one by one: off by less than one step of the block's last scale (integers), or 2^-4 of a value
    and a step below the normal ones (floats)."""
    g = np.random.default_rng(1)
    codes, scales = np.zeros((1, 1, 16, 8), np.uint8), np.zeros((1, 1, 1), np.float32)
    x = (g.standard_normal((16, 1, 8)) * np.exp(g.uniform(-3, 3, (16, 1, 1)))).astype(np.float32)
    for t in range(16):
        ref.append(codes, scales, x[t:t + 1], np.array([0, 1]), np.array([t]), np.zeros((1, 1), int), 16, kind)
    got = ref.values(codes[0, 0], kind) * float(scales[0, 0, 0])
    off, s = np.abs(got - x[:, 0]), float(scales[0, 0, 0])
    if kind == "i8":
        assert (off < s).all() and s * 127 < 2 * np.abs(x).max() * (1 + 1e-6)
    else:
        assert (off <= np.maximum(np.abs(x[:, 0]) * 2.0 ** -4, s * 2.0 ** -9)).all()
