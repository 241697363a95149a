"""GPU tests of attention over an 8-bit cache where a tolerance does not notice: what no row sees, bit for bit."""
import numpy as np
import pytest

import compensated_fp32_projection_amd as cf
from gpu_helpers import note
from test_attention8_gpu import problem
from test_cache8_gpu import cache_of, dev, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("lens,Hq,Hkv,D,page,block", [([37, 5, 0, 64, 90], 8, 2, 64, 16, 4), ([33, 2, 130], 4, 4, 128, 64, 16),
                                                      ([19, 700], 3, 1, 40, 16, 1), ([9, 21], 6, 2, 64, 4, 2)])
@pytest.mark.parametrize("unseen", [np.inf, -np.inf, np.nan, 2.0 ** 127, 0.0])
def test_unseen_scales_change_no_bit(unseen, lens, Hq, Hkv, D, page, block, kind):
    """Scales of blocks behind the last token are 1, and then what memory may hold: the results are the same bits."""
    rng = np.random.default_rng(D + page)
    q, arrays, table, lens = problem(rng, lens, Hq, Hkv, D, page, block, kind)
    seen = np.zeros((len(arrays[1]), page // block), bool)
    for b, n in enumerate(lens):
        for j in range(n):
            seen[table[b, j // page], j % page // block] = True
    got = []
    for value in (1.0, unseen):
        for i in (1, 3):
            arrays[i][~seen[:, None, :].repeat(Hkv, 1)] = value
        c, *_ = cache_of(arrays, kind)
        note(f"decode8 unseen bits {lens} {D} {page} {block} {kind} {value}")
        got += host(cf.attention8_decode(dev(q), c, dev(table), dev(lens)))
    assert np.array_equal(got[0], got[1])
