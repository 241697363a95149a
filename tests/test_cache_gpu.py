"""GPU tests of the paged cache's calls against plain bookkeeping: whole
results, every count and every byte of the pools."""
import numpy as np
import pytest
import torch

import attention_reference as ref
import compensated_fp32_projection_amd as cf
from gpu_helpers import note

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(*ts):
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in ts]


def pools(rng, P, Hkv, page, D, kv):
    dt = np.float16 if kv == "f16" else np.float32
    return [rng.standard_normal((P, Hkv, page, D), dtype=np.float32).astype(dt) for _ in range(2)]


def placed(x, layout):
    """A device copy of a pool in another layout of the same shape."""
    t = dev(x)
    if layout == "token_major":
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "odd_offset":
        return torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)
    if layout == "padded":
        P, H, n, D = t.shape
        return torch.zeros((P, H + 1, n + 1, D + 3), dtype=t.dtype, device="cuda")[:, :H, :n, :D].copy_(t)
    return t


def tables(rng, S, W, page, P, spare=0):
    """Distinct pages for S sequences of random lengths (some 0, some whole pages), and the counts."""
    lens = rng.integers(0, W * page + 1, S)
    lens[rng.random(S) < 0.2] = 0
    lens = np.where(rng.random(S) < 0.3, lens // page * page, lens)
    ids = rng.permutation(P)[:P - spare]
    table, at = np.full((S, W), -1, np.int32), 0
    for s in range(S):
        m = -(-int(lens[s]) // page)
        if at + m > len(ids):
            m = 0
            lens[s] = 0
        table[s, :m] = ids[at:at + m]
        at += m
    refs = np.zeros(P, np.int32)
    refs[table[table >= 0]] = 1
    return table, lens.astype(np.int32), refs


# pool sizes up to more free pages than one pass over the pool lists (8192)
@pytest.mark.parametrize("P,S,W,page,grow", [(1, 1, 1, 16, 3), (7, 3, 4, 1, 2), (64, 5, 9, 16, 60), (300, 20, 12, 8, 50),
                                             (5000, 64, 40, 16, 900), (30000, 400, 60, 4, 300), (0, 2, 3, 4, 5)])
@pytest.mark.parametrize("in_place", [False, True])
def test_reserve(P, S, W, page, grow, in_place):
    rng = np.random.default_rng(P + S)
    note(f"reserve {P} {S} {W} {page}")
    table, lens, refs = tables(rng, S, W, page, P)
    cu = np.concatenate([[0], np.cumsum(rng.integers(0, grow + 1, S))]).astype(np.int32)
    want_t, want_r, missing = ref.reserve(table, lens, refs, cu, page)
    t, r, m = dev(table), dev(refs), torch.full((1,), 99, dtype=torch.int32, device="cuda")
    kw = dict(table_out=t, refs_out=r) if in_place else {}
    got = host(*cf.cache_reserve(t, dev(lens), r, dev(cu), page, missing=m, **kw), m)
    assert np.array_equal(got[0], want_t) and np.array_equal(got[1], want_r) and got[2][0] == missing
    if not in_place:
        assert np.array_equal(*host(t, dev(table))) and np.array_equal(*host(r, dev(refs)))


def test_reserve_a_view_of_a_wider_table():
    rng = np.random.default_rng(3)
    table, lens, refs = tables(rng, 6, 5, 8, 60)
    wide = np.full((6, 9), 77, np.int32)
    wide[:, 2:7] = table
    cu = (np.arange(7) * 5).astype(np.int32)
    want_t, want_r, _ = ref.reserve(table, lens, refs, cu, 8)
    t, r = dev(wide), dev(refs)
    note("reserve view")
    cf.cache_reserve(t[:, 2:7], dev(lens), r, dev(cu), 8, table_out=t[:, 2:7], refs_out=r)
    got, got_r = host(t, r)
    assert np.array_equal(got[:, 2:7], want_t) and np.array_equal(got_r, want_r)
    assert (got[:, :2] == 77).all() and (got[:, 7:] == 77).all()


@pytest.mark.parametrize("kv", ["f32", "f16"])
@pytest.mark.parametrize("layout", ["plain", "token_major", "odd_offset", "padded"])
@pytest.mark.parametrize("S,page,Hkv,D,new", [(1, 16, 8, 128, [1]), (5, 4, 2, 64, [0, 1, 9, 0, 30]), (70, 16, 1, 10, [1] * 70),
                                              (3, 1, 3, 7, [4, 4, 4])])
def test_append(S, page, Hkv, D, new, layout, kv):
    rng = np.random.default_rng(S + D)
    note(f"append {S} {page} {Hkv} {D} {layout} {kv}")
    P, W = 40 + S * 10, 12
    table, lens, refs = tables(rng, S, 4, page, P)
    table = np.pad(table, ((0, 0), (0, W - 4)), constant_values=-1)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    table, refs, _ = ref.reserve(table, lens, refs, cu, page)
    k_pages, v_pages = pools(rng, P, Hkv, page, D, kv)
    k, v = (rng.standard_normal((cu[-1], Hkv, D), dtype=np.float32) * 3 for _ in range(2))
    k.reshape(-1)[:3] = [1e-7, 65504.0, 1.0 + 2.0 ** -11]  # a subnormal, the largest and a tie of FP16
    tk, tv = placed(k_pages, layout), placed(v_pages, layout)
    got_lens, = host(cf.cache_append(dev(k), dev(np.repeat(v, 2, 0))[::2], dev(cu), tk, tv, dev(table), dev(lens)))
    want_lens = ref.append(k, v, cu, k_pages, v_pages, table, lens)
    got_k, got_v = host(tk, tv)
    assert np.array_equal(got_lens, want_lens)
    assert np.array_equal(got_k, k_pages) and np.array_equal(got_v, v_pages)


def test_append_leaves_bad_places_alone():
    """Tokens past the table, in entries of -1 or of no page, or before 0."""
    rng = np.random.default_rng(4)
    k_pages, v_pages = pools(rng, 6, 2, 4, 8, "f32")
    table = np.array([[0, -1, 2], [99, 3, -7], [4, 5, 1]], np.int32)
    lens = np.array([2, 0, -3], np.int32)
    cu = np.array([0, 15, 25, 32], np.int32)
    k, v = (rng.standard_normal((40, 2, 8), dtype=np.float32) for _ in range(2))
    tk, tv = dev(k_pages), dev(v_pages)
    note("append bad places")
    cf.cache_append(dev(k), dev(v), dev(cu), tk, tv, dev(table), dev(lens))
    ref.append(k, v, cu, k_pages, v_pages, table, lens)
    got = host(tk, tv)
    assert np.array_equal(got[0], k_pages) and np.array_equal(got[1], v_pages)


@pytest.mark.parametrize("kv", ["f32", "f16"])
@pytest.mark.parametrize("layout", ["plain", "token_major", "odd_offset", "padded"])
@pytest.mark.parametrize("Hkv,page,D", [(8, 16, 128), (3, 4, 10), (1, 1, 1), (2, 64, 64)])
def test_copy_pages(Hkv, page, D, layout, kv):
    rng = np.random.default_rng(page + D)
    note(f"copy {Hkv} {page} {D} {layout} {kv}")
    k_pages, v_pages = pools(rng, 20, Hkv, page, D, kv)
    src, dst = np.array([3, 3, 19, -1, 0, 7], np.int32), np.array([4, 5, 6, 8, 20, 2], np.int32)
    tk, tv = placed(k_pages, layout), placed(v_pages, layout)
    cf.cache_copy_pages(tk, tv, dev(src), dev(dst))
    for a, b in ((3, 4), (3, 5), (19, 6), (7, 2)):
        k_pages[b], v_pages[b] = k_pages[a], v_pages[a]
    got = host(tk, tv)
    assert np.array_equal(got[0], k_pages) and np.array_equal(got[1], v_pages)


# parents: some several times, one outside the table; pools with room and without
@pytest.mark.parametrize("P,S,W,page,C,spare", [(64, 1, 8, 16, 4, 20), (200, 12, 10, 8, 60, 90), (100, 9, 9, 4, 50, 3),
                                                (12000, 30, 20, 2, 9000, 9500), (4, 1, 1, 4, 0, 2)])
@pytest.mark.parametrize("in_place", [False, True])
def test_fork(P, S, W, page, C, spare, in_place):
    rng = np.random.default_rng(P + C)
    note(f"fork {P} {S} {W} {page} {C}")
    table, lens, refs = tables(rng, S, W, page, P, spare)
    k_pages, v_pages = pools(rng, P, 2, page, 8, "f16")
    parents = rng.integers(0, S, C).astype(np.int32)
    if C > 10:
        parents[[2, 7]] = [-1, S]
    tk, tv, r = dev(k_pages), dev(v_pages), dev(refs)
    m = torch.full((1,), 99, dtype=torch.int32, device="cuda")
    got = host(*cf.cache_fork(tk, tv, dev(table), dev(lens), r, dev(parents), missing=m,
                              refs_out=r if in_place else None), m, tk, tv)
    t2, r2, l2, missing = ref.fork(k_pages, v_pages, table, lens, refs, parents)
    for a, b in zip(got, (t2, r2, l2, [missing], k_pages, v_pages)):
        assert np.array_equal(a, b)


def test_fork_of_broken_tables():
    """Entries of -1 and ids outside the pool are inherited and counted nowhere;
    a last page that is none is not copied."""
    rng = np.random.default_rng(5)
    k_pages, v_pages = pools(rng, 10, 1, 4, 8, "f32")
    table = np.array([[0, -1, 99, 3], [4, -1, -1, -1], [5, 6, -1, -1]], np.int32)
    lens, refs = np.array([15, 6, 99], np.int32), np.ones(10, np.int32)
    refs[[7, 8]] = [0, -2]
    parents = np.array([0, 1, 2, 0], np.int32)
    tk, tv = dev(k_pages), dev(v_pages)
    note("fork broken tables")
    got = host(*cf.cache_fork(tk, tv, dev(table), dev(lens), dev(refs), dev(parents)), tk, tv)
    t2, r2, l2, _ = ref.fork(k_pages, v_pages, table, lens, refs, parents)
    for a, b in zip(got, (t2, r2, l2, k_pages, v_pages)):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("P,R,W", [(1, 1, 1), (50, 0, 4), (50, 7, 9), (40000, 300, 500)])
@pytest.mark.parametrize("in_place", [False, True])
def test_free(P, R, W, in_place):
    rng = np.random.default_rng(P + R)
    rows = rng.integers(-3, P + 3, (R, W)).astype(np.int32)
    refs = rng.integers(0, 5, P).astype(np.int32)
    r = dev(refs)
    note(f"free {P} {R} {W}")
    got, = host(cf.cache_free(dev(rows), r, refs_out=r if in_place else None))
    assert np.array_equal(got, ref.free(rows, refs))


@pytest.mark.parametrize("P,live", [(1, 0), (1, 1), (2, 1), (100, 0), (100, 100), (100, 37), (1025, 600), (9000, 4000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(P, live, in_place):
    rng = np.random.default_rng(P + live)
    note(f"compact {P} {live}")
    refs = np.zeros(P, np.int32)
    refs[rng.permutation(P)[:live]] = rng.integers(1, 4, live)
    refs[(refs == 0) & (rng.random(P) < 0.1)] = -1
    table = rng.integers(-1, P + 2, (9, 17)).astype(np.int32)
    named = (table >= 0) & (table < P)
    table[named & (refs[np.where(named, table, 0)] <= 0)] = -1  # tables name live pages
    k_pages, v_pages = pools(rng, P, 2, 4, 8, "f16")
    tk, tv, t, r = dev(k_pages), dev(v_pages), dev(table), dev(refs)
    kw = dict(table_out=t, refs_out=r) if in_place else {}
    got = host(*cf.cache_compact(tk, tv, t, r, **kw), tk, tv)
    t2, r2, n = ref.compact(k_pages, v_pages, table, refs)
    for a, b in zip(got, (t2, r2, [n], k_pages, v_pages)):
        assert np.array_equal(a, b)


def test_graph_of_a_serving_step():
    """Reserve, append, fork, free and compact captured once; every replay on
    new counts equals the eager calls."""
    rng = np.random.default_rng(6)
    P, S, W, page = 200, 8, 10, 8
    table, lens, refs = tables(rng, S, 6, page, P)
    table = np.pad(table, ((0, 0), (0, W - 6)), constant_values=-1)
    k_pages, v_pages = pools(rng, P, 2, page, 16, "f16")
    cu = (np.arange(S + 1) * 3).astype(np.int32)
    k, v = (dev(rng.standard_normal((3 * S, 2, 16), dtype=np.float32)) for _ in range(2))
    t, l, r, c, p = dev(table), dev(lens), dev(refs), dev(cu), dev(np.array([0, 3, 3, 7], np.int32))
    tk, tv = dev(k_pages), dev(v_pages)

    def step(stream=None, ws=None):
        t1, r1 = cf.cache_reserve(t, l, r, c, page, stream=stream)
        l1 = cf.cache_append(k, v, c, tk, tv, t1, l, stream=stream)
        t2, r2, l2 = cf.cache_fork(tk, tv, t1, l1, r1, p, workspace=ws, stream=stream)
        r3 = cf.cache_free(t1[:4], r2, stream=stream)
        both = torch.cat([t1[4:], t2])
        return (*cf.cache_compact(tk, tv, both, r3, workspace=ws, stream=stream), l2)

    note("cache graph")
    ws = cf.Workspace()
    step(ws=ws)
    tk.copy_(dev(k_pages))
    tv.copy_(dev(v_pages))
    torch.cuda.synchronize()
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(st):
        with torch.cuda.graph(g, stream=st):
            outs = step(stream=st, ws=ws)
    torch.cuda.synchronize()
    for i in range(4):
        k.copy_(torch.randn_like(k))
        table2, lens2, refs2 = tables(rng, S, 6, page, P)
        t.copy_(dev(np.pad(table2, ((0, 0), (0, W - 6)), constant_values=-1)))
        l.copy_(dev(lens2))
        r.copy_(dev(refs2))
        tk.copy_(dev(k_pages))
        tv.copy_(dev(v_pages))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = host(*outs, tk, tv)
        tk.copy_(dev(k_pages))
        tv.copy_(dev(v_pages))
        want = host(*step(), tk, tv)
        for a, b in zip(got, want):
            assert np.array_equal(a, b), f"replay {i}"
