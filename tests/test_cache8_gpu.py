"""GPU tests of the 8-bit cache against its definition: every code and scale of
the pools, and every value read back, bit for bit."""
import numpy as np
import pytest
import torch

import attention_reference as paged
import cache8_reference as ref
import compensated_fp32_projection_amd as cf
from gpu_helpers import note

pytestmark = pytest.mark.gpu

DTYPE = {"i8": torch.int8, "e4m3": torch.float8_e4m3fn}


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(*ts):
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in ts]


def tables(rng, S, W, page, P, pages):
    """Distinct pages, `pages[s]` of them for sequence s."""
    ids, table, at = rng.permutation(P), np.full((S, W), -1, np.int32), 0
    for s in range(S):
        table[s, :pages[s]] = ids[at:at + pages[s]]
        at += pages[s]
    return table


def pools(rng, P, H, page, D, block, kind):
    """Codes (bytes) and scales of K and V; float scales are powers of two."""
    out = []
    for _ in range(2):
        codes = rng.integers(-127, 128, (P, H, page, D)).astype(np.int8).view(np.uint8) if kind == "i8" else \
            ref.nearest(rng.standard_normal((P, H, page, D)) * 100, kind)
        scales = np.exp(rng.uniform(-5, 0, (P, H, page // block)))
        out += [codes, (scales if kind == "i8" else 2.0 ** np.floor(np.log2(scales))).astype(np.float32)]
    return out


def placed(x, layout):
    """A device copy in another layout of the same shape."""
    t = dev(x)
    if layout == "token_major" and t.dim() == 4:
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if layout == "odd":
        return torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)
    if layout == "padded":
        return torch.zeros([n + 1 for n in t.shape[:-1]] + [t.shape[-1] + 3], dtype=t.dtype,
                           device="cuda")[tuple(slice(0, n) for n in t.shape)].copy_(t)
    return t


def cache_of(arrays, kind, layout="plain"):
    """A Cache8 of numpy codes and scales (K, then V), and its code tensors as bytes."""
    codes = [placed(a, layout) for a in arrays[::2]]
    scales = [placed(a, layout) for a in arrays[1::2]]
    views = [c.view(DTYPE[kind]) for c in codes]
    return cf.Cache8(*views, *scales), codes[0], scales[0], codes[1], scales[1]


def same(got, want):
    for a, b in zip(got, want):
        assert a.dtype == b.dtype and a.shape == b.shape
        if a.dtype == np.float32:
            bad = ~((a.view(np.uint32) == b.view(np.uint32)) | (np.isnan(a) & np.isnan(b)))
        elif a.dtype == np.float16:
            bad = ~((a.view(np.uint16) == b.view(np.uint16)) | (np.isnan(a) & np.isnan(b)))
        else:
            bad = a != b
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), a[bad][:4], b[bad][:4])


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("layout", ["plain", "token_major", "odd", "padded"])
@pytest.mark.parametrize("page,block,H,D,lens,new", [
    (16, 16, 8, 128, [5], [1]),
    (16, 16, 3, 64, [0, 1, 15, 16, 17, 31, 40], [1, 1, 1, 1, 1, 1, 1]),
    (32, 8, 2, 40, [0, 3, 8, 30, 64], [0, 1, 9, 40, 70]),
    (4, 1, 2, 10, [0, 3, 4], [5, 1, 9]),
    (1, 1, 1, 7, [2, 0], [3, 4]),
    (128, 128, 2, 80, [0, 100, 127, 128], [300, 27, 2, 128]),
    (64, 2, 1, 1, [1, 63], [64, 2]),
    (16, 4, 2, 128, [2] * 70, [1, 0] * 35),
])
def test_append(page, block, H, D, lens, new, layout, kind):
    rng = np.random.default_rng(page + D)
    note(f"append8 {page} {block} {H} {D} {layout} {kind}")
    S, lens = len(lens), np.array(lens, np.int32)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    pages = [-(-(int(a) + b) // page) for a, b in zip(lens, new)]
    P, W = sum(pages) + 3, max(pages) + 1
    table = tables(rng, S, W, page, P, pages)
    arrays = pools(rng, P, H, page, D, block, kind)
    # Magnitudes over several powers of two, so that blocks grow by none, one and more.
    k, v = (((rng.standard_normal((cu[-1], H, D)) * np.exp(rng.uniform(-6, 6, (cu[-1], H, 1))))).astype(np.float32)
            for _ in range(2))
    c, *parts = cache_of(arrays, kind, layout)
    got_lens, = host(cf.cache8_append(dev(k), dev(np.repeat(v, 2, 0))[::2], dev(cu), c, dev(table), dev(lens)))
    assert np.array_equal(got_lens, lens + np.diff(cu))
    for codes, scales, x in ((arrays[0], arrays[1], k), (arrays[2], arrays[3], v)):
        ref.append(codes, scales, x, cu, lens, table, block, kind)
    same(host(*parts), arrays)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_a_block_filled_token_by_token(kind):
    """Growth after growth, with all that a block's codes can be, and a value on every border."""
    rng = np.random.default_rng(3)
    page = block = 32
    arrays = pools(rng, 2, 2, page, 16, block, kind)
    table = np.array([[1]], np.int32)
    c, *parts = cache_of(arrays, kind)
    note(f"append8 token by token {kind}")
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu, t = dev(np.array([0, 1], np.int32)), dev(table)
    for i in range(page):
        k, v = ((rng.standard_normal((1, 2, 16)) * 2.0 ** rng.uniform(-8 + i / 2, -6 + i / 2)).astype(np.float32) for _ in range(2))
        for x, s in ((k, arrays[1]), (v, arrays[3])):
            if i:  # halves and whole steps of the scale there is
                x[0, :, :8] = np.array([0.5, 1.5, 2.5, -0.5, 126.5, -3.5, 1, 0])[None] * s[1, :, 0][:, None]
        lens = cf.cache8_append(dev(k), dev(v), cu, c, t, lens)
        for codes, scales, x in ((arrays[0], arrays[1], k), (arrays[2], arrays[3], v)):
            ref.append(codes, scales, x, [0, 1], [i], table, block, kind)
        same(host(*parts), arrays)
    assert int(lens) == page


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_quotients_next_to_ties(kind):
    """Values whose quotient by the scale is a half and a last bit more or less."""
    rng = np.random.default_rng(8)
    D = 128
    arrays = pools(rng, 8, 1, 16, D, 16, kind)
    table = np.arange(8, dtype=np.int32).reshape(8, 1)
    lens, cu = np.full(8, 1, np.int32), np.arange(9, dtype=np.int32)
    x = np.zeros((8, 1, D), np.float32)
    for s in range(8):
        step = arrays[1][s, 0, 0]
        half = ((np.arange(D) % 120 + 0.5) * np.float64(step)).astype(np.float32)
        x[s, 0] = np.nextafter(half, np.where(np.arange(D) % 3 == 0, 0, np.where(np.arange(D) % 3 == 1, np.inf, half))
                               .astype(np.float32)) * (-1) ** s
    c, *parts = cache_of(arrays, kind)
    note(f"append8 ties {kind}")
    cf.cache8_append(dev(x), dev(x), dev(cu), c, dev(table), dev(lens))
    ref.append(arrays[0], arrays[1], x, cu, lens, table, 16, kind)
    ref.append(arrays[2], arrays[3], x, cu, lens, table, 16, kind)
    same(host(*parts), arrays)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_extreme_values(kind):
    """Zeros, subnormals, the largest finite values, infinities and NaN, in new blocks and in begun ones."""
    rng = np.random.default_rng(9)
    big = np.finfo(np.float32).max
    rows = [[0, 0, 0, 0], [-0.0, 0, 0, 0], [1e-45, 0, -1e-45, 3e-39], [1.2e-38, -1e-38, 5e-39, 1e-40], [big, -big, 1, 0],
            [np.inf, 1, 2, 3], [1, -np.inf, 0, 0], [np.nan, 1, 2, 3], [448, 449, 0.25, 1e-3], [127, 127.4, 63.5, 64.5]]
    x = np.array(rows, np.float32)[:, None, :].repeat(2, 1)
    S = len(rows)
    for begun in (0, 3):
        arrays = pools(rng, S, 2, 8, 4, 8, kind)
        if begun:
            for s, bad in enumerate([np.nan, np.inf, 0.0, -1.0, 1e-39]):  # scales that are none
                arrays[1][s] = arrays[3][s] = bad
        table, lens = np.arange(S, dtype=np.int32).reshape(S, 1), np.full(S, begun, np.int32)
        cu = np.arange(S + 1, dtype=np.int32)
        c, *parts = cache_of(arrays, kind)
        note(f"append8 extremes {kind} {begun}")
        cf.cache8_append(dev(x), dev(x[::-1]), dev(cu), c, dev(table), dev(lens))
        ref.append(arrays[0], arrays[1], x, cu, lens, table, 8, kind)
        ref.append(arrays[2], arrays[3], x[::-1], cu, lens, table, 8, kind)
        same(host(*parts), arrays)
    assert np.isnan(arrays[1]).any() and np.isfinite(arrays[1]).any()


def test_append_leaves_bad_places_alone():
    """Tokens past the table, in entries of -1 or of no page, of a negative length, and rows outside all sequences."""
    rng = np.random.default_rng(4)
    arrays = pools(rng, 6, 2, 4, 8, 2, "i8")
    table = np.array([[0, -1, 2], [99, 3, -7], [4, 5, 1]], np.int32)
    lens, cu = np.array([2, 0, -3], np.int32), np.array([3, 15, 25, 32], np.int32)
    k, v = (rng.standard_normal((40, 2, 8)).astype(np.float32) for _ in range(2))
    c, *parts = cache_of(arrays, "i8")
    note("append8 bad places")
    got, = host(cf.cache8_append(dev(k), dev(v), dev(cu), c, dev(table), dev(lens)))
    assert np.array_equal(got, lens + np.diff(cu))
    ref.append(arrays[0], arrays[1], k, cu, lens, table, 2, "i8")
    ref.append(arrays[2], arrays[3], v, cu, lens, table, 2, "i8")
    same(host(*parts), arrays)
    # No tokens, no pages, offsets that are none: nothing is written, and nothing faults.
    for cu2 in ([0, 0, 0, 0], [-5, -2, 1, 1], [50, 60, 70, 1 << 30], [9, 4, 2, 0]):
        lens2 = np.array([0, 0, 0], np.int32)
        before = host(*parts)
        got, = host(cf.cache8_append(dev(k[:0]), dev(v[:0]), dev(np.array(cu2, np.int32)), c, dev(table), dev(lens2)))
        assert np.array_equal(got, np.diff(np.array(cu2)))
        same(host(*parts), before)
    empty = cf.Cache8.empty(0, 2, 4, 8)
    cf.cache8_append(dev(k), dev(v), dev(cu), empty, dev(table), dev(lens))
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("dtype", [np.float32, np.float16])
@pytest.mark.parametrize("layout", ["plain", "token_major", "odd", "padded"])
@pytest.mark.parametrize("page,block,H,D,counts", [(16, 16, 8, 128, [1]), (8, 2, 3, 40, [0, 5, 1, 0, 17]), (64, 32, 2, 64, [130, 64]),
                                                   (4, 1, 1, 7, [9, 3]), (16, 8, 2, 1, [20]), (32, 32, 12, 80, [300, 1, 2])])
def test_read(page, block, H, D, counts, layout, dtype, kind):
    rng = np.random.default_rng(page + D)
    note(f"read8 {page} {block} {H} {D} {layout} {dtype} {kind}")
    S = len(counts)
    first = rng.integers(0, 2 * page, S).astype(np.int32)
    pages = [-(-(int(a) + b) // page) for a, b in zip(first, counts)]
    P = sum(pages) + 2
    table = tables(rng, S, max(pages) + 1, page, P, pages)
    arrays = pools(rng, P, H, page, D, block, kind)
    cu = np.concatenate([[2], 2 + np.cumsum(counts)]).astype(np.int32)  # two rows before the first sequence
    T = int(cu[-1]) + 3                                                # and three behind the last
    c, *_ = cache_of(arrays, kind, layout)
    want = [ref.read(arrays[i], arrays[i + 1], cu, first, table, block, kind, np.full((T, H, D), 7, dtype), dtype)
            for i in (0, 2)]
    outs = [placed(np.full((T, H, D), 7, dtype), "plain" if layout == "token_major" else layout) for _ in range(2)]
    got = cf.cache8_read(c, dev(table), dev(cu), T, first=dev(first), dtype=outs[0].dtype, k_out=outs[0], v_out=outs[1])
    same(host(*got), want)


def test_read_of_every_code_and_of_places_that_are_none():
    codes = np.arange(256, dtype=np.uint8).reshape(1, 1, 4, 64).repeat(3, 0)
    table = np.array([[0, -1, 2, 9], [2, 1, 0, 0]], np.int32)
    cu, first = np.array([0, 20, 40], np.int32), np.array([-2, 3], np.int32)
    for kind in ("i8", "e4m3"):
        scales = np.array([0.1, np.nan, 3e38], np.float32).reshape(3, 1, 1)
        c, *_ = cache_of([codes, scales, codes[::-1].copy(), scales], kind)
        note(f"read8 every code {kind}")
        for dtype, kt in ((np.float32, torch.float32), (np.float16, torch.float16)):
            with np.errstate(over="ignore"):
                want = ref.read(codes, scales, cu, first, table, 4, kind, np.zeros((40, 1, 64), dtype), dtype)
            same(host(cf.cache8_read(c, dev(table), dev(cu), 40, first=dev(first), dtype=kt)[0]), [want])
    assert np.isnan(want[:2]).all()
    none = cf.Cache8.empty(0, 1, 4, 64)
    assert bool(torch.isnan(cf.cache8_read(none, dev(table), dev(cu), 40)[0]).all())


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("layout", ["plain", "token_major", "odd", "padded"])
@pytest.mark.parametrize("H,page,block,D", [(8, 16, 16, 128), (3, 4, 2, 10), (1, 1, 1, 1), (2, 64, 8, 65)])
def test_pages_are_moved_with_their_scales(H, page, block, D, layout, kind):
    rng = np.random.default_rng(page + D)
    note(f"move8 {H} {page} {D} {layout} {kind}")
    P, S, W = 40, 4, 5
    arrays = pools(rng, P, H, page, D, block, kind)
    c, *parts = cache_of(arrays, kind, layout)
    src, dst = np.array([3, 3, 19, -1, 0, 7], np.int32), np.array([4, 5, 6, 8, 40, 2], np.int32)
    cf.cache8_copy_pages(c, dev(src), dev(dst))
    for a in arrays:
        for i, j in ((3, 4), (3, 5), (19, 6), (7, 2)):
            a[j] = a[i]
    same(host(*parts), arrays)

    lens = rng.integers(1, W * page + 1, S).astype(np.int32)
    table = tables(rng, S, W, page, P, [-(-int(n) // page) for n in lens])
    refs = np.zeros(P, np.int32)
    refs[table[table >= 0]] = 1
    parents = np.array([0, 2, 2, -1, 3], np.int32)
    m = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    t, r, n = cf.cache8_fork(c, dev(table), dev(lens), dev(refs), dev(parents), missing=m)
    t2, r2, l2, missing = paged.fork(arrays[0], arrays[2], table, lens, refs, parents)
    fork_scales(arrays, table, lens, refs, parents, page)
    same(host(t, r, n, m, *parts), [t2, r2, l2, np.array([missing], np.int32), *arrays])

    kept = np.concatenate([t2, table[:1]])
    r3 = paged.free(table[1:], r2)
    t, r, live = cf.cache8_compact(c, dev(kept), dev(r3))
    t4, r4, n4 = paged.compact(arrays[0], arrays[2], kept, r3)
    paged.compact(arrays[1], arrays[3], kept, r3)
    same(host(t, r, live, *parts), [t4, r4, np.array([n4], np.int32), *arrays])


def fork_scales(arrays, table, lens, refs, parents, page):
    """The copies of a fork, of scales: a page's scales go with its codes."""
    free = [p for p, n in enumerate(refs) if n <= 0]
    for p in parents:
        if 0 <= p < len(lens) and lens[p] % page:
            to = free.pop(0)
            for a in (arrays[1], arrays[3]):
                a[to] = a[table[p, lens[p] // page]]


def test_the_class_refuses():
    ok = lambda: [torch.zeros(3, 2, 16, 8, dtype=torch.int8, device="cuda") for _ in range(2)] + \
        [torch.zeros(3, 2, 4, device="cuda") for _ in range(2)]
    c = cf.Cache8(*ok())
    assert c.block == 4 and c.shape == (3, 2, 16, 8)
    for i, bad in ((0, torch.zeros(3, 2, 16, 8, device="cuda")), (1, torch.zeros(3, 2, 16, 9, dtype=torch.int8, device="cuda")),
                   (1, torch.zeros(3, 2, 16, 8, dtype=torch.float8_e4m3fn, device="cuda")),
                   (0, torch.zeros(3, 2, 8, 16, dtype=torch.int8, device="cuda").transpose(2, 3)),
                   (2, torch.zeros(3, 2, 3, device="cuda")), (3, torch.zeros(3, 2, 4, dtype=torch.float64, device="cuda")),
                   (2, torch.zeros(2, 2, 4, device="cuda")), (2, torch.zeros(3, 2, 16, 8)),
                   (3, torch.zeros(3, 4, 2, device="cuda").transpose(1, 2))):
        args = ok()
        args[i] = bad
        with pytest.raises((TypeError, ValueError)):
            cf.Cache8(*args)
    with pytest.raises(ValueError):
        cf.Cache8(*(torch.zeros(3, 2, 6, 8, dtype=torch.int8, device="cuda") for _ in range(2)),
                  *(torch.zeros(3, 2, 2, device="cuda") for _ in range(2)))
    with pytest.raises(ValueError):
        cf.Cache8.empty(3, 2, 16, 8, block=5)
    assert cf.Cache8.empty(3, 2, 16, 8, block=8, dtype=torch.float8_e4m3fn).k.dtype == torch.float8_e4m3fn


def test_other_streams_and_a_graph():
    """Written and read on another stream, and captured: every replay on new tokens is the eager call's result."""
    rng = np.random.default_rng(11)
    P, H, page, D, S = 24, 2, 16, 64, 4
    arrays = pools(rng, P, H, page, D, 8, "i8")
    lens, cu = np.array([3, 0, 20, 8], np.int32), np.array([0, 5, 6, 20, 24], np.int32)
    table = tables(rng, S, 4, page, P, [3] * 4)
    x = [dev(rng.standard_normal((24, H, D)).astype(np.float32)) for _ in range(2)]
    t, ln, c_, all_ = dev(table), dev(lens), dev(cu), dev(np.arange(5, dtype=np.int32) * 30)

    def step(c, stream=None):
        n = cf.cache8_append(x[0], x[1], c_, c, t, ln, stream=stream)
        return (n, *cf.cache8_read(c, t, all_, 120, stream=stream))

    note("cache8 streams and graph")
    c1, *parts1 = cache_of(arrays, "i8")
    want = host(*step(c1), *parts1)
    c2, *parts2 = cache_of(arrays, "i8")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = step(c2, st)
    same(host(*got, *parts2), want)
    c3, *parts3 = cache_of(arrays, "i8")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(g, stream=st):
            outs = step(c3, st)
    for i in range(3):
        for y in x:
            y.mul_(1.5)
        for part, a in zip(parts3, arrays):
            part.copy_(dev(a))
        torch.cuda.synchronize()
        g.replay()
        got = host(*outs, *parts3)
        c4, *parts4 = cache_of(arrays, "i8")
        same(got, host(*step(c4), *parts4))


def test_pools_beyond_32_bits():
    """Codes and scales more than 2^32 elements behind the pools' beginnings."""
    stride = (1 << 31) + 64
    note("cache8 large strides")
    base = torch.zeros(2 * stride + 16 * 64, dtype=torch.int8, device="cuda")
    k = base.as_strided((3, 1, 16, 64), (stride, 16 * 64, 64, 1))
    v = torch.zeros(3, 1, 16, 64, dtype=torch.int8, device="cuda")
    sc = [torch.zeros(3, 1, 2, device="cuda") for _ in range(2)]
    c = cf.Cache8(k, v, *sc)
    x = torch.randn(16, 1, 64, device="cuda")
    t = torch.tensor([[2]], dtype=torch.int32, device="cuda")
    cu, zero = dev(np.array([0, 16], np.int32)), dev(np.array([0], np.int32))
    cf.cache8_append(x, x, cu, c, t, zero)
    a, b = cf.cache8_read(c, t, cu, 16)
    assert torch.equal(a, b) and torch.equal(k[2], v[2]) and bool((a != 0).any()) and not bool(k[0].any() | k[1].any())
