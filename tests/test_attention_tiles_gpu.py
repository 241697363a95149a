"""GPU tests of the attention calls at sizes that go through 64-key tiles in LDS
(many rows: long or many prompts, prefixes shared by more than 32 rows),
against the definition in FP64 (tolerance derived in attention_reference.py).
Some K/V heads of each case are compared, all of their query heads."""
import numpy as np
import pytest
import torch

import attention_reference as ref
import compensated_fp32_projection_amd as cf
from gpu_helpers import note
from test_attention_decode_gpu import call as decode_call
from test_attention_decode_gpu import make as decode_make
from test_attention_prompt_gpu import call, check, dev, make, starts

pytestmark = pytest.mark.gpu


def compare(got, q, k, v, cu_q, cu_k, heads, causal=True, scale=None, what="", rows=slice(None)):
    """The K/V heads `heads` of a prompt's result."""
    g = q.shape[1] // k.shape[1]
    for j in heads:
        hs = slice(j * g, j * g + g)
        want, bound, written = ref.prompt(q[:, hs], k[:, j:j + 1], v[:, j:j + 1], cu_q, cu_k, causal, scale)
        check(got[:, hs][rows], want[rows], bound[rows], f"{what} K/V head {j}")


CASES = [
    # query rows, keys, Hq, Hkv, D, kv, causal, heads compared
    ([1100], [1100], 12, 12, 64, "f32", True, [0, 11]),
    ([1089], [1153], 12, 12, 64, "f32", True, [5]),                 # 17 tiles before, an odd number of them
    ([250, 350], [250, 350], 32, 8, 128, "f32", True, [0, 7]),
    ([250, 350], [250, 350], 32, 8, 128, "f32", False, [3]),
    ([129, 0, 1, 400, 63], [193, 0, 65, 400, 64], 32, 8, 128, "f32", True, [2]),
    ([300, 290, 310], [300, 400, 350], 16, 8, 80, "f32", True, [6]),
    ([700, 500], [700, 500], 9, 3, 40, "f32", True, [1]),
    ([1500], [1500], 12, 12, 64, "f32", True, [4]),                 # keys in parts
    ([1600], [1600], 12, 12, 64, "f16", True, [7]),
    ([100, 120, 90, 110], [100, 120, 90, 110], 32, 8, 128, "f16", True, [0, 7]),
    ([100, 120, 90, 110], [10, 320, 0, 110], 32, 8, 128, "f16", True, [1]),  # rows that see nothing
    ([128] * 8, [128] * 8, 16, 2, 64, "f16", True, [0, 1]),
    ([120, 127, 129, 128] * 3, [120, 127, 129, 128] * 3, 14, 2, 64, "f16", False, [1]),
    ([300, 200, 250], [310, 264, 250], 16, 16, 80, "f16", True, [9]),
    ([400, 300, 200, 350, 450, 300, 250, 350], [400, 364, 200, 350, 450, 300, 250, 350], 32, 8, 128, "f16", True, [6]),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}h{c[2]}-{c[3]}d{c[4]}{c[5]}{'' if c[6] else 'all'}")
def test_prompts(case):
    lq, lk, Hq, Hkv, D, kv, causal, heads = case
    note(f"tiles prompt {lq} {lk} {Hq}/{Hkv} x {D} {kv} causal={causal}")
    q, k, v = make(sum(lk) + D, lq, lk, Hq, Hkv, D, kv)
    cu_q, cu_k = starts(lq), starts(lk)
    compare(call(dev(q), dev(k), dev(v), cu_q, cu_k, causal=causal), q, k, v, cu_q, cu_k, heads, causal)


@pytest.mark.parametrize("layout", ["head_major", "padded_rows", "odd_offset", "large_strides"])
@pytest.mark.parametrize("kv", ["f32", "f16"])
def test_layouts(layout, kv):
    """Strides of every kind; what does not allow 16-byte loads of FP16 keys goes
    the other way, with the same result."""
    Hq, Hkv, D = (12, 12, 64) if kv == "f32" else (32, 8, 128)
    lens = [1100] if kv == "f32" else [100, 110, 120, 100]
    note(f"tiles layout {layout} {kv}")
    q, k, v = make(31, lens, lens, Hq, Hkv, D, kv)
    T = sum(lens)
    tq, tk, tv, out = dev(q), dev(k), dev(v), None
    if layout == "head_major":
        tq, tk, tv = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (tq, tk, tv))
        out = torch.full((Hq, T, D), 7.0, device="cuda").transpose(0, 1)
    elif layout == "padded_rows":
        def pad(x):
            y = torch.full((T, x.shape[1] + 1, D + 8), float("nan"), dtype=x.dtype, device="cuda")
            y[:, :x.shape[1], :D] = x
            return y[:, :x.shape[1], :D]
        tq, tk, tv, out = pad(tq), pad(tk), pad(tv), pad(torch.full((T, Hq, D), 7.0, device="cuda"))
    elif layout == "odd_offset":
        def off(x):
            return torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(x.shape).copy_(x)
        tq, tk, tv, out = off(tq), off(tk), off(tv), off(torch.full((T, Hq, D), 7.0, device="cuda"))
    else:  # the last keys more than 2^32 bytes from the first
        def far(x):
            stride = (1 << 33) // (x.element_size() * T) // 8 * 8
            return torch.empty((T - 1) * stride + x.shape[1] * D, dtype=x.dtype, device="cuda").as_strided(
                x.shape, (stride, D, 1)).copy_(x)
        tk, tv = far(tk), far(tv)
    cu = starts(lens)
    compare(call(tq, tk, tv, cu, cu, out=out), q, k, v, cu, cu, [Hkv - 1], what=layout)


@pytest.mark.parametrize("kv", ["f32", "f16"])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_what_is_masked_does_not_matter(kv, bad):
    """One bad value among those that some rows of a tile see and others do not,
    and all of another sequence's."""
    Hq, Hkv, D = (12, 12, 64) if kv == "f32" else (32, 8, 128)
    lens, at = ([1000, 150, 60], 700) if kv == "f32" else ([200, 150, 120], 90)
    note(f"tiles masked {bad} {kv}")
    q, k, v = make(32, lens, lens, Hq, Hkv, D, kv)
    cu = starts(lens)
    g, j = Hq // Hkv, 1
    hs = slice(j * g, j * g + g)
    want, bound, _ = ref.prompt(q[:, hs], k[:, j:j + 1], v[:, j:j + 1], cu, cu)
    v[at, :, 7] = bad
    k[cu[1]:cu[2]] = bad
    v[cu[1]:cu[2]] = bad
    got = call(dev(q), dev(k), dev(v), cu, cu)[:, hs]
    check(got[:at], want[:at], bound[:at], "rows before it")
    keep = np.arange(D) != 7
    check(got[at:cu[1]][..., keep], want[at:cu[1]][..., keep], bound[at:cu[1]][..., keep], "beside it")
    assert (np.isnan(got[at:cu[1], :, 7]) if np.isnan(bad) else got[at:cu[1], :, 7] == bad).all()
    assert not np.isfinite(got[cu[1]:cu[2]]).any()
    check(got[cu[2]:], want[cu[2]:], bound[cu[2]:], "the next sequence")


@pytest.mark.parametrize("sq,sk,sv", [(1e-20, 1e20, 1.0), (1e18, 1e-18, 1e30), (1.0, 1.0, 1e-30), (3e4, 1e-5, 7e4)])
def test_ranges_of_fp32(sq, sk, sv):
    note(f"tiles ranges {sq} {sk} {sv}")
    q, k, v = make(33, [1050], [1050], 12, 12, 64, "f32")
    q, k, v = (x * np.float32(f) for x, f in ((q, sq), (k, sk), (v, sv)))
    cu = starts([1050])
    compare(call(dev(q), dev(k), dev(v), cu, cu), q, k, v, cu, cu, [8])


def test_values_of_very_different_tiles():
    """Value magnitudes that change by powers of 2^20 from tile to tile, tiles of zeros among them."""
    rng = np.random.default_rng(34)
    T, H, D = 1088, 12, 64
    q, k, v = make(34, [T], [T], H, H, D, "f32")
    f = np.float32(2.0) ** (20 * rng.integers(-2, 3, T // 64)).astype(np.float32)
    f[[0, 5, 9]] = 0
    v *= f.repeat(64)[:, None, None]
    cu = starts([T])
    note("tiles of different magnitude")
    got = call(dev(q), dev(k), dev(v), cu, cu)
    assert (got[:64] == 0).all()
    compare(got, q, k, v, cu, cu, [3], rows=slice(64, None))


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_scale(scale):
    note(f"tiles scale {scale}")
    lens = [100, 110, 120, 100]
    q, k, v = make(35, lens, lens, 32, 8, 128, "f16")
    cu = starts(lens)
    compare(call(dev(q), dev(k), dev(v), cu, cu, scale=scale), q, k, v, cu, cu, [2], scale=scale)


@pytest.mark.parametrize("kv", ["f32", "f16"])
def test_graph_replays_and_streams(kv):
    """The same bits eagerly, on a side stream, and from a graph on new inputs and offsets."""
    Hq, Hkv, D = (12, 12, 64) if kv == "f32" else (32, 8, 128)
    T = 1500 if kv == "f32" else 460
    q, k, v = (dev(x) for x in make(36, [T], [T], Hq, Hkv, D, kv))
    cu = dev(starts([T // 2, T - T // 2]))
    note(f"tiles graph {kv}")
    a = cf.attention_prompt(q, k, v, cu)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    b = cf.attention_prompt(q, k, v, cu, stream=side, workspace=cf.Workspace())
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    out, ws = torch.empty_like(q), cf.Workspace()
    cf.attention_prompt(q, k, v, cu, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            cf.attention_prompt(q, k, v, cu, out=out, workspace=ws, stream=side)
    torch.cuda.synchronize()
    for r in range(3):
        q.copy_(torch.randn_like(q))
        cu.copy_(dev(starts([T // 5 * (r + 1), T - T // 5 * (r + 1)])))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, cf.attention_prompt(q, k, v, cu)), f"replay {r}"


DECODES = [
    # lens, shared pages, page, Hq, Hkv, D
    ([700 + 3 * i for i in range(40)], 10, 64, 4, 1, 128),        # 160 rows, two blocks
    ([1030] * 9, 1024, 1, 8, 2, 64),                              # a page for each token
    ([600, 640, 641, 3, 0, 512, 700, 100, 639], 10, 64, 16, 2, 80),  # lengths that end inside the prefix
    ([512] * 12, 2, 256, 4, 1, 64),                               # nothing beyond the prefix
    ([1000 + i for i in range(17)], 62, 16, 14, 2, 64),
    ([90, 80, 100, 70, 95, 85, 75, 99, 64], 1, 64, 32, 8, 128),   # one tile
]


@pytest.mark.parametrize("case", DECODES, ids=lambda c: f"{len(c[0])}x{max(c[0])}s{c[1]}p{c[2]}h{c[3]}-{c[4]}d{c[5]}")
def test_shared_prefixes(case):
    lens, shared, page, Hq, Hkv, D = case
    note(f"tiles decode {case}")
    q, k, v, table, lens = decode_make(sum(lens) + D, lens, shared, page, Hq, Hkv, D, "f16")
    want, bound = ref.decode(q, k, v, table, lens)
    check(decode_call(dev(q), dev(k), dev(v), table, lens, shared_pages=shared), want, bound)


def test_bad_pages_and_values_in_a_shared_prefix():
    """A bad page id in the prefix makes NaN of the rows that reach it, an
    infinite value reaches those that see it, and what lies beyond a length
    does not matter."""
    lens = [200 + 60 * (i % 8) for i in range(24)]
    q, k, v, table, lens = decode_make(41, lens, 6, 64, 8, 2, 64, "f16")
    want, bound = ref.decode(q, k, v, table, lens)
    note("tiles bad pages in a prefix")
    t = table.copy()
    t[:, 5] = 10 ** 6
    got = decode_call(dev(q), dev(k), dev(v), t, lens, shared_pages=6)
    hit = lens > 5 * 64
    assert hit.any() and not hit.all() and np.isnan(got[hit]).all()
    check(got[~hit], want[~hit], bound[~hit], "rows that do not reach the page")
    v[table[0, 4], :, 10, 5] = np.inf
    got = decode_call(dev(q), dev(k), dev(v), table, lens, shared_pages=6)
    see, keep = lens > 4 * 64 + 10, np.arange(64) != 5
    assert (got[see][..., 5] == np.inf).all()
    check(got[see][..., keep], want[see][..., keep], bound[see][..., keep], "beside the infinity")
    check(got[~see], want[~see], bound[~see], "rows that do not see it")


def test_long_shared_prefix_keeps_its_precision():
    """2^16 keys: sums over many parts stay FP32-grade."""
    note("tiles decode of 65536 shared keys")
    B, Hq, Hkv, D, page = 12, 4, 1, 64, 64
    rng = np.random.default_rng(42)
    n = 1 << 16
    k, v = (rng.standard_normal((n // page + B, Hkv, page, D), dtype=np.float32).astype(np.float16) for _ in range(2))
    q = rng.standard_normal((B, Hq, D), dtype=np.float32)
    table = np.concatenate([np.arange(n // page, dtype=np.int32)[None].repeat(B, 0),
                            (n // page + np.arange(B, dtype=np.int32))[:, None]], axis=1)
    lens = np.full(B, n + 5, np.int32)
    want, bound = ref.decode(q, k, v, table, lens)
    check(decode_call(dev(q), dev(k), dev(v), table, lens, shared_pages=n // page), want, bound)


LONG_DECODES = [
    # lens, shared pages, page, Hq, Hkv, D: many rows behind a long prefix
    ([5952 + 3 * i for i in range(20)], 93, 64, 64, 8, 128),
    ([6030 + i for i in range(40)], 6000, 1, 32, 8, 128),                     # a page for each token
    ([6000, 6400, 6401, 3, 0, 5120, 7000, 1000, 6399, 64] * 2, 400, 16, 64, 8, 80),  # lengths that end inside the prefix
    ([6144] * 20, 24, 256, 64, 8, 128),                                       # nothing beyond the prefix
    ([12100 + 7 * i for i in range(30)], 378, 32, 14, 2, 64),
]


@pytest.mark.parametrize("case", LONG_DECODES, ids=lambda c: f"{len(c[0])}x{max(c[0])}s{c[1]}p{c[2]}h{c[3]}-{c[4]}d{c[5]}")
def test_long_shared_prefixes(case):
    lens, shared, page, Hq, Hkv, D = case
    note(f"tiles decode {len(lens)}x{max(lens)} shared {shared} of {page} {Hq}/{Hkv} x {D}")
    q, k, v, table, lens = decode_make(sum(lens) + D, lens, shared, page, Hq, Hkv, D, "f16")
    got = decode_call(dev(q), dev(k), dev(v), table, lens, shared_pages=shared)
    g = Hq // Hkv
    for j in (0, Hkv - 1):
        hs = slice(j * g, j * g + g)
        want, bound = ref.decode(q[:, hs], k[:, j:j + 1], v[:, j:j + 1], table, lens)
        check(got[:, hs], want, bound, f"K/V head {j}")


def test_bad_pages_and_values_in_a_long_shared_prefix():
    lens = [5000 + 300 * (i % 8) for i in range(24)]
    Hq, Hkv, page, shared = 64, 8, 64, 96
    q, k, v, table, lens = decode_make(43, lens, shared, page, Hq, Hkv, 128, "f16")
    hs = slice(8, 16)
    want, bound = ref.decode(q[:, hs], k[:, 1:2], v[:, 1:2], table, lens)
    note("tiles bad pages in a long prefix")

    def run(t):
        return decode_call(dev(q), dev(k), dev(v), t, lens, shared_pages=shared)[:, hs]

    t = table.copy()
    t[:, 90] = -7
    got, hit = run(t), lens > 90 * page
    assert hit.any() and not hit.all() and np.isnan(got[hit]).all()
    check(got[~hit], want[~hit], bound[~hit], "rows that do not reach the page")
    v[table[0, 85], :, 10, 5] = np.inf
    v[table[0, 95]] = np.nan
    got, see, lost = run(table), lens > 85 * page + 10, lens > 95 * page
    assert np.isnan(got[lost]).all() and (got[see & ~lost][..., 5] == np.inf).all()
    keep = np.arange(128) != 5
    rest = see & ~lost
    check(got[rest][..., keep], want[rest][..., keep], bound[rest][..., keep], "beside the infinity")
    check(got[~see], want[~see], bound[~see], "rows that do not see it")


def test_long_shared_prefix_repeats():
    """The same bits every time, on a side stream with its own workspace, and from a graph as sequences grow."""
    q, k, v, table, lens = (dev(x) for x in decode_make(44, [6200] * 20, 90, 64, 64, 8, 128, "f16", unused=0))
    note("tiles decode repeats")
    a = cf.attention_decode(q, k, v, table, lens, shared_pages=90)
    torch.cuda.synchronize()
    side, ws = torch.cuda.Stream(), cf.Workspace()
    b = cf.attention_decode(q, k, v, table, lens, shared_pages=90, stream=side, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            cf.attention_decode(q, k, v, table, lens, shared_pages=90, out=out, workspace=ws, stream=side)
    torch.cuda.synchronize()
    for r in range(3):
        lens -= 100
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, cf.attention_decode(q, k, v, table, lens, shared_pages=90)), f"replay {r}"
