"""GPU tests of the cache calls on a pool of 2^31 - 1 pages (of one value each):
loops over pages and counts end within 32 bits."""
import pytest
import torch

import compensated_fp32_projection_amd as cf
from gpu_helpers import note

pytestmark = pytest.mark.gpu

P = 2 ** 31 - 1


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_free_and_reserve():
    refs = torch.ones(P, dtype=torch.int32, device="cuda")
    refs[-3:] = 0
    note("free of 2^31 - 1 pages")
    out = cf.cache_free(ints(P - 5, 0, P - 1, P - 5)[None], refs)
    torch.cuda.synchronize()
    assert out[[0, 1, P - 5, P - 4, P - 1]].tolist() == [0, 1, -1, 1, -1]
    out[[0, P - 5, P - 1]] = refs[[0, P - 5, P - 1]]
    assert torch.equal(out, refs)
    del out
    note("reserve of 2^31 - 1 pages")
    missing = ints(0)
    table, out = cf.cache_reserve(ints(7, -1, -1, -1)[None], ints(1), refs, ints(0, 10), page=2, missing=missing)
    torch.cuda.synchronize()
    assert table.tolist() == [[7, P - 3, P - 2, P - 1]] and missing.tolist() == [2]
    assert out[-4:].tolist() == [1, 1, 1, 1]
    out[-3:] = 0
    assert torch.equal(out, refs)


def test_fork_and_compact():
    refs = torch.ones(P, dtype=torch.int32, device="cuda")
    refs[[3, P - 4]] = 0
    pools = [torch.zeros(P, 1, 1, 1, dtype=torch.float16, device="cuda") for _ in range(2)]
    for x in pools:
        x[P - 1] = 5
    note("fork of 2^31 - 1 pages")
    table, out, lens = cf.cache_fork(*pools, ints(P - 1, 1, P - 2, -1)[None], ints(3), refs, ints(0, 0))
    torch.cuda.synchronize()
    assert table.tolist() == [[P - 1, 1, P - 2, -1]] * 2 and lens.tolist() == [3, 3]
    assert out[[1, P - 2, P - 1, 0, P - 4]].tolist() == [3, 3, 3, 1, 0]
    del out
    note("compaction of 2^31 - 1 pages")
    table, out, live = cf.cache_compact(*pools, ints(P - 1, 1, P - 2, -1)[None], refs)
    torch.cuda.synchronize()
    # P - 2 live pages: those at P - 2 and P - 1 move into the free ones below.
    assert live.tolist() == [P - 2] and table.tolist() == [[P - 4, 1, 3, -1]]
    assert out[[3, P - 4, P - 3, P - 2, P - 1]].tolist() == [1, 1, 1, 0, 0]
    assert [float(x[P - 4]) for x in pools] == [5, 5]
    assert int(out.sum()) == P - 2
