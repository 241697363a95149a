"""GPU tests of the prompt attention at sizes whose blocks have eight waves
(more than 1024 blocks of 128 rows and long sequences; FP32 K and V with heads
over 64 from 512 on), against the definition in FP64 for some K/V heads."""
import numpy as np
import pytest

import attention_reference as ref
from gpu_helpers import note
from test_attention_prompt_gpu import call, check, dev, make, starts
from test_attention_tiles_gpu import compare

pytestmark = pytest.mark.gpu

CASES = [
    # query rows, keys, Hq, Hkv, D, kv, causal, heads compared
    ([1200, 1150], [1200, 1281], 64, 16, 128, "f16", True, [0, 15]),
    ([1200, 1150], [1281, 1150], 64, 16, 72, "f16", False, [7]),
    ([1153, 0, 1290, 1], [1153, 500, 1290, 1500], 64, 16, 64, "f16", True, [3]),
    ([1200, 1150], [1200, 1281], 64, 16, 64, "f32", True, [15]),
    ([1177, 1190], [300, 2100], 64, 16, 40, "f32", True, [2]),      # rows that see nothing
    ([290, 310, 270, 300, 305, 295, 340, 290], [290, 374, 270, 300, 305, 295, 340, 290], 32, 8, 128, "f32", True, [5]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}h{c[2]}-{c[3]}d{c[4]}{c[5]}{'' if c[6] else 'all'}")
def test_prompts(case):
    lq, lk, Hq, Hkv, D, kv, causal, heads = case
    note(f"long tiles prompt {lq} {lk} {Hq}/{Hkv} x {D} {kv} causal={causal}")
    q, k, v = make(sum(lk) + D, lq, lk, Hq, Hkv, D, kv)
    cu_q, cu_k = starts(lq), starts(lk)
    compare(call(dev(q), dev(k), dev(v), cu_q, cu_k, causal=causal), q, k, v, cu_q, cu_k, heads, causal)


@pytest.mark.parametrize("kv", ["f32", "f16"])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_what_is_masked_does_not_matter(kv, bad):
    """A bad value that a sequence's last rows see."""
    note(f"long tiles masked {bad} {kv}")
    lens, at = [1200, 1190], 1100
    q, k, v = make(41, lens, lens, 64, 16, 64, kv)
    cu = starts(lens)
    hs = slice(4, 8)
    want, bound, _ = ref.prompt(q[:, hs], k[:, 1:2], v[:, 1:2], cu, cu)
    v[at, 1, 5] = bad
    got = call(dev(q), dev(k), dev(v), cu, cu)[:, hs]
    check(got[:at], want[:at], bound[:at], "rows before it")
    keep = np.arange(64) != 5
    check(got[at:cu[1]][..., keep], want[at:cu[1]][..., keep], bound[at:cu[1]][..., keep], "beside it")
    seen = got[at:cu[1], :, 5]
    assert (np.isnan(seen) if np.isnan(bad) else seen == bad).all()
    check(got[cu[1]:], want[cu[1]:], bound[cu[1]:], "the next sequence")
