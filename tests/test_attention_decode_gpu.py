"""GPU tests of cfp32_attention_decode against the definition in FP64 (tolerance
derived in attention_reference.py): lengths around page and tile edges, shared
prefixes of many rows, pages of every size, what unused places hold, bad page
ids, strides, streams and graphs."""
import numpy as np
import pytest
import torch

import attention_reference as ref
import compensated_fp32_projection_amd as cf
from gpu_helpers import note
from test_attention_prompt_gpu import check, dev

pytestmark = pytest.mark.gpu


def make(seed, lens, shared, page, Hq, Hkv, D, kv, extra_width=0, unused=np.nan):
    """q, pools, table, lens: pages in random order, `unused` wherever no sequence has a token."""
    rng = np.random.default_rng(seed)
    B = len(lens)
    W = max(shared, max(-(-n // page) for n in lens)) + extra_width
    own = [[j for j in range(shared, -(-n // page))] for n in lens]
    P = shared + sum(map(len, own)) + 3
    ids = rng.permutation(P).astype(np.int32)
    table = np.full((B, W), -1, np.int32)
    table[:, :shared] = ids[:shared]
    at = shared
    dt = np.float16 if kv == "f16" else np.float32
    k, v = (np.full((P, Hkv, page, D), unused, dt) for _ in range(2))
    for x in (k, v):
        x[ids[:shared]] = rng.standard_normal((shared, Hkv, page, D), dtype=np.float32)
    for b, n in enumerate(lens):
        for j in own[b]:
            table[b, j] = ids[at]
            m = min(page, n - j * page)
            for x in (k, v):
                x[ids[at], :, :m] = rng.standard_normal((Hkv, m, D), dtype=np.float32)
            at += 1
    q = rng.standard_normal((B, Hq, D), dtype=np.float32) * 1.5
    return q, k, v, table, np.asarray(lens, np.int32)


def call(q, k, v, table, lens, **kw):
    o = cf.attention_decode(q, k, v, dev(table), dev(lens), **kw)
    torch.cuda.synchronize()
    return o.cpu().numpy()


CASES = [
    # lens, shared pages, page, Hq, Hkv, D
    ([1], 0, 16, 4, 2, 64),
    ([130], 0, 16, 32, 8, 128),
    ([0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65], 0, 16, 4, 2, 64),
    ([0, 0], 0, 16, 2, 1, 64),
    ([127, 128, 129, 300], 0, 64, 8, 2, 128),
    ([5, 9, 40], 0, 1, 4, 1, 64),                          # a page for each token
    ([5, 300, 256, 257, 513], 0, 256, 4, 4, 128),
    ([64 + 5, 64, 64 + 200, 64 + 1], 1, 64, 4, 2, 128),    # one that ends with the prefix
    ([500, 481, 600, 480, 499], 30, 16, 12, 12, 64),       # a prefix that ends inside a tile
    ([2100 + i for i in range(40)], 32, 64, 8, 2, 64),     # 160 rows per K/V head
    ([1300] * 3, 20, 64, 32, 2, 128),                      # 48 rows per K/V head
    ([700, 3, 0, 640, 641, 100], 10, 64, 4, 2, 64),        # lengths that end inside the prefix
    ([3000, 10], 0, 32, 2, 1, 40),
    ([90, 33], 2, 16, 9, 3, 63),
    ([70, 66], 1, 64, 3, 3, 1),
]


@pytest.mark.parametrize("kv", ["f32", "f16"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}s{c[1]}p{c[2]}h{c[3]}-{c[4]}d{c[5]}")
def test_lengths_and_pages(case, kv):
    lens, shared, page, Hq, Hkv, D = case
    note(f"decode {case} {kv}")
    q, k, v, table, lens = make(sum(lens) + D, lens, shared, page, Hq, Hkv, D, kv)
    want, bound = ref.decode(q, k, v, table, lens)
    for s in {0, shared, max(0, shared - 1)}:
        check(call(dev(q), dev(k), dev(v), table, lens, shared_pages=s), want, bound, f"shared {s}")


@pytest.mark.parametrize("kv", ["f32", "f16"])
@pytest.mark.parametrize("layout", ["token_major", "odd_offset", "padded", "strided_q", "wide_table"])
def test_layouts(layout, kv):
    note(f"decode layout {layout} {kv}")
    q, k, v, table, lens = make(21, [200, 170, 161], 2, 32, 8, 2, 64, kv, extra_width=3 if layout == "wide_table" else 0)
    want, bound = ref.decode(q, k, v, table, lens)
    tq, tk, tv, kw = dev(q), dev(k), dev(v), {}
    if layout == "token_major":
        tk, tv = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (tk, tv))
    elif layout == "odd_offset":
        def off(x):
            return torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(x.shape).copy_(x)
        tq, tk, tv = off(tq), off(tk), off(tv)
    elif layout == "padded":
        def pad(x):
            y = torch.full((x.shape[0], 3, 33, 67), float("nan"), dtype=x.dtype, device="cuda")
            y[:, :2, :32, :64] = x
            return y[:, :2, :32, :64]
        tk, tv = pad(tk), pad(tv)
    elif layout == "strided_q":
        tq = dev(np.repeat(q, 2, axis=0))[::2]
        kw["out"] = torch.full((8, 3, 64), 7.0, device="cuda").transpose(0, 1)
    check(call(tq, tk, tv, table, lens, shared_pages=2, **kw), want, bound, layout)


@pytest.mark.parametrize("kv", ["f32", "f16"])
@pytest.mark.parametrize("bad", [-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1])
def test_bad_page_ids_are_not_read(bad, kv):
    """A page id outside the pool where a sequence has tokens makes its row NaN
    and no other; one it does not need is not looked at."""
    note(f"decode bad page {bad} {kv}")
    q, k, v, table, lens = make(22, [200, 170, 161, 190], 2, 32, 4, 2, 64, kv, extra_width=2)
    want, bound = ref.decode(q, k, v, table, lens)
    table[0, 4] = bad
    table[1:, 7] = bad
    got = call(dev(q), dev(k), dev(v), table, lens, shared_pages=2)
    assert np.isnan(got[0]).all()
    check(got[1:], want[1:], bound[1:])


def test_lens_outside_the_table_are_clamped():
    q, k, v, table, lens = make(23, [96, 64], 0, 32, 4, 2, 64, "f16")
    table[1, 2] = table[1, 1]
    full = np.array([96, 96], np.int32)
    want, bound = ref.decode(q, k, v, table, full)
    note("decode lens outside the table")
    check(call(dev(q), dev(k), dev(v), table, np.array([2 ** 31 - 1, 97], np.int32)), want, bound)
    assert (call(dev(q), dev(k), dev(v), table, np.array([-5, -2 ** 31], np.int32)) == 0).all()


@pytest.mark.parametrize("sq,sk,sv", [(1e-20, 1e20, 1.0), (1e18, 1e-18, 1e30), (1.0, 1.0, 1e-30)])
def test_ranges_of_fp32(sq, sk, sv):
    note(f"decode ranges {sq} {sk} {sv}")
    q, k, v, table, lens = make(24, [300, 250], 3, 64, 4, 2, 64, "f32", unused=0)
    q, k, v = (x * np.float32(f) for x, f in ((q, sq), (k, sk), (v, sv)))
    want, bound = ref.decode(q, k, v, table, lens)
    check(call(dev(q), dev(k), dev(v), table, lens, shared_pages=3), want, bound)


@pytest.mark.parametrize("kv", ["f32", "f16"])
def test_visible_infinities(kv):
    """An infinite value a sequence sees reaches its row; a NaN key makes the row NaN."""
    q, k, v, table, lens = make(25, [200, 170], 0, 32, 4, 2, 64, kv)
    want, bound = ref.decode(q, k, v, table, lens)
    v[table[0, 1], :, 3, 5] = np.inf
    k[table[1, 2], :, 1, 0] = np.nan
    note(f"decode infinities {kv}")
    got = call(dev(q), dev(k), dev(v), table, lens)
    assert (got[0, :, 5] == np.inf).all() and np.isnan(got[1]).all()
    keep = np.arange(64) != 5
    check(got[:1][..., keep], want[:1][..., keep], bound[:1][..., keep])


def test_offsets_beyond_32_bits():
    """Pages more than 2^32 bytes apart."""
    q, k, v, table, lens = make(26, [100, 90], 1, 32, 2, 1, 64, "f16", unused=0)
    P, stride = k.shape[0], (1 << 30) + 64
    note("decode large offsets")
    def far(x):
        y = torch.empty((P - 1) * stride + 32 * 64, dtype=torch.float16, device="cuda")
        return y.as_strided((P, 1, 32, 64), (stride, 32 * 64, 64, 1)).copy_(dev(x))
    want, bound = ref.decode(q, k, v, table, lens)
    check(call(dev(q), far(k), far(v), table, lens, shared_pages=1), want, bound)


def test_repeats_and_other_stream():
    q, k, v, table, lens = (dev(x) for x in make(27, [1500] * 6, 20, 64, 8, 2, 128, "f16"))
    a = cf.attention_decode(q, k, v, table, lens, shared_pages=20)
    torch.cuda.synchronize()
    b = cf.attention_decode(q, k, v, table, lens, shared_pages=20, stream=torch.cuda.Stream(), workspace=cf.Workspace())
    c = cf.attention_decode(q, k, v, table, lens, shared_pages=20)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)


def test_graph_replays():
    """Captured once, replayed as the sequences grow."""
    q, k, v, table, _ = make(28, [400, 400, 400], 4, 32, 4, 2, 64, "f16", unused=0)
    q, k, v, table = dev(q), dev(k), dev(v), dev(table)
    lens, ws = dev(np.array([140, 150, 160], np.int32)), cf.Workspace()
    out = torch.empty_like(q)
    note("decode graph")
    cf.attention_decode(q, k, v, table, lens, shared_pages=4, out=out, workspace=ws)
    torch.cuda.synchronize()
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(st):
        with torch.cuda.graph(g, stream=st):
            cf.attention_decode(q, k, v, table, lens, shared_pages=4, out=out, workspace=ws, stream=st)
    torch.cuda.synchronize()
    for r in range(4):
        lens += 50
        q.copy_(torch.randn_like(q))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want = cf.attention_decode(q, k, v, table, lens, shared_pages=4, workspace=cf.Workspace())
        assert torch.equal(got, want), f"replay {r}"
