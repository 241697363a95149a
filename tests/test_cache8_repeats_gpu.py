"""GPU tests of the 8-bit cache where later tokens are as large as those that made a block's scale."""
import numpy as np
import pytest
import torch

import compensated_fp32_projection_amd as cf
from gpu_helpers import note
from test_cache8_gpu import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("D", [16, 7])
def test_a_repeated_token_leaves_the_scale(D, dtype):
    """The same token again, of 8000 largest magnitudes over all of FP32's range: scales and codes stay, and the new
    token's codes are the first one's."""
    S, H = 1000, 8
    rng = np.random.default_rng(D)
    x = (rng.uniform(-1, 1, (2, S, H, D)) * 2.0 ** rng.integers(-120, 120, (2, S, H, 1))).astype(np.float32)
    c = cf.Cache8.empty(S, H, 4, D, dtype=dtype)
    table = dev(np.arange(S, dtype=np.int32)[:, None])
    lens, cu = dev(np.zeros(S, np.int32)), dev(np.arange(S + 1, dtype=np.int32))
    k, v = dev(x[0]), dev(x[1])
    note(f"cache8 repeats {D} {dtype}")
    lens = cf.cache8_append(k, v, cu, c, table, lens)
    ks, vs = c.k_scales.clone(), c.v_scales.clone()
    for _ in range(3):
        lens = cf.cache8_append(k, v, cu, c, table, lens)
    assert torch.equal(c.k_scales, ks) and torch.equal(c.v_scales, vs)
    for codes in (c.k, c.v):
        codes = codes.view(torch.uint8)
        assert all(torch.equal(codes[:, :, i], codes[:, :, 0]) for i in range(1, 4))
    assert int(lens.min()) == 4


def test_what_a_scale_held_before_it_still_holds():
    """Scales of other origin: a token whose largest magnitude is 127 scales, in FP32, leaves them."""
    S, H, D = 1000, 8, 8
    rng = np.random.default_rng(1)
    s = (rng.uniform(1, 2, (S, H, 1)) * 2.0 ** rng.integers(-100, 100, (S, H, 1))).astype(np.float32)
    c = cf.Cache8.empty(S, H, 4, D)
    c.k_scales.copy_(dev(s))
    c.v_scales.copy_(dev(s))
    x = np.zeros((S, H, D), np.float32)
    x[..., 3] = s[..., 0] * np.float32(127)
    table = dev(np.arange(S, dtype=np.int32)[:, None])
    note("cache8 held before")
    cf.cache8_append(dev(x), dev(-x), dev(np.arange(S + 1, dtype=np.int32)), c, table, dev(np.ones(S, np.int32)))
    assert torch.equal(c.k_scales, dev(s)) and torch.equal(c.v_scales, dev(s))
    assert bool((c.k[:, :, 1, 3] == 127).all()) and bool((c.v[:, :, 1, 3] == -127).all())
