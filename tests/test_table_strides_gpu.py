"""GPU tests of tables whose rows are one (expanded): what only reads a table takes them, what writes pages or counts
refuses them."""
import numpy as np
import pytest
import torch

import attention_reference as paged
import cache8_reference as ref
import compensated_fp32_projection_amd as cf
import test_attention8_gpu as att8
from gpu_helpers import note
from test_cache8_gpu import cache_of, dev, host

pytestmark = pytest.mark.gpu


def one_row(rng, lens, Hq, Hkv, D, kind):
    """Sequences of different lengths in the pages of the longest."""
    q, arrays, table, _ = att8.problem(rng, [max(lens)], Hq, Hkv, D, 16, 8, kind)
    q = rng.standard_normal((len(lens), Hq, D)).astype(np.float32)
    return q, arrays, table, np.array(lens, np.int32)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("lens", [[50, 3, 0, 64], [3000, 2999, 17]])
def test_the_8_bit_cache(lens, kind):
    rng = np.random.default_rng(1)
    q, arrays, table, lens = one_row(rng, lens, 4, 2, 64, kind)
    c, *_ = cache_of(arrays, kind)
    t = dev(table).expand(len(lens), table.shape[1])
    want = att8.expected(q, arrays, kind, 8, np.repeat(table, len(lens), 0), lens)
    note(f"decode8 one row {lens} {kind}")
    att8.check(cf.attention8_decode(dev(q), c, t, dev(lens)), want)
    att8.check(cf.attention8_decode(dev(q), c, t, dev(lens), workspace=cf.Workspace()), want)  # without the native form
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    n = int(cu[-1])
    got = cf.cache8_read(c, t, dev(cu), n)
    outs = [torch.empty_like(x) for x in got]
    cf.cache8_read(c, t, dev(cu), n, k_out=outs[0], v_out=outs[1])
    for i, pair in enumerate(zip(host(*got), host(*outs))):
        out = ref.read(arrays[2 * i], arrays[2 * i + 1], cu, None, np.repeat(table, len(lens), 0), 8, kind,
                       np.zeros(pair[0].shape, np.float32), np.float32)
        assert np.array_equal(pair[0], out) and np.array_equal(pair[1], out)


@pytest.mark.parametrize("shared", [0, 2])
def test_the_paged_cache(shared):
    rng = np.random.default_rng(2)
    lens, page, Hq, Hkv, D = np.array([100, 40, 64, 33], np.int32), 16, 8, 2, 64
    k, v = (rng.standard_normal((9, Hkv, page, D)).astype(np.float32) for _ in range(2))
    q = rng.standard_normal((4, Hq, D)).astype(np.float32)
    table = rng.permutation(9)[None, :7].astype(np.int32)
    out, bound = paged.decode(q, k.astype(np.float64), v.astype(np.float64), np.repeat(table, 4, 0), lens, D ** -0.5)
    note(f"decode one row {shared}")
    t = dev(table).expand(4, 7)
    for kw in ({}, dict(workspace=cf.Workspace())):
        got, = host(cf.attention_decode(dev(q), dev(k), dev(v), t, dev(lens), shared_pages=shared, **kw))
        assert (np.abs(got - out) <= bound).all()


def test_what_writes_refuses_them():
    c = cf.Cache8.empty(8, 2, 16, 64)
    pools = [torch.zeros(8, 2, 16, 64, device="cuda") for _ in range(2)]
    t = torch.zeros(1, 3, dtype=torch.int32, device="cuda").expand(2, 3)
    lap = torch.zeros(9, dtype=torch.int32, device="cuda").as_strided((2, 3), (2, 1))
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    cu, refs = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(8, dtype=torch.int32, device="cuda")
    x, q = torch.zeros(0, 2, 64, device="cuda"), torch.zeros(2, 4, 64, device="cuda")
    for bad in (t, lap):
        for f in (lambda: cf.cache_reserve(bad, i, refs, cu, 16), lambda: cf.cache_append(x, x, cu, *pools, bad, i),
                  lambda: cf.cache_fork(*pools, bad, i, refs, i), lambda: cf.cache_free(bad, refs),
                  lambda: cf.cache_compact(*pools, bad, refs), lambda: cf.cache8_append(x, x, cu, c, bad, i),
                  lambda: cf.cache8_fork(c, bad, i, refs, i), lambda: cf.cache8_compact(c, bad, refs)):
            with pytest.raises(ValueError, match="overlap"):
                f()
    for f in (lambda: cf.attention8_decode(q, c, lap, i), lambda: cf.cache8_read(c, lap, cu, 1),
              lambda: cf.attention_decode(q, *pools, lap, i)):
        with pytest.raises(ValueError, match="overlap"):
            f()
