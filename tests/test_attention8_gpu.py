"""GPU tests of attention over an 8-bit cache against FP64 on the values that its
codes and scales stand for.

The bound is attention_reference's, whose terms cover the split of q, the sums
and the exponential (a score is scaled by two factors more, a weight by one: 6 e
of those it allows for splitting K and the weights), and one term more: a product
of a weight and V's scale is off by 2^-36 of the largest of its step at the most,
times a code of 448 at most: 2^-36 n max_j(w_j s_j) 448 / sum_j w_j.
"""
import numpy as np
import pytest
import torch

import attention_reference as paged
import cache8_reference as ref
import compensated_fp32_projection_amd as cf
from gpu_helpers import note
from test_cache8_gpu import cache_of, dev, host, placed, pools, tables

pytestmark = pytest.mark.gpu


def expected(q, arrays, kind, block, table, lens, scale=None):
    k, v = (ref.values(arrays[i], kind) * np.repeat(arrays[i + 1].astype(np.float64), block, axis=2)[..., None] for i in (0, 2))
    B, Hq, D = q.shape
    g = Hq // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out, bound = paged.decode(q, k, v, table, lens, scale)
    for b in range(B):
        n = int(lens[b])
        if not n:
            continue
        kb = paged.gather(k, table[b], n)
        sb = paged.gather(np.repeat(np.abs(arrays[3].astype(np.float64)), block, axis=2)[..., None], table[b], n)[..., 0]
        for h in range(Hq):
            s = scale * (kb[:, h // g] @ q[b, h].astype(np.float64))
            w = np.exp(s - s.max())
            bound[b, h] += 2.0 ** -36 * n * (w * sb[:, h // g]).max() * ref.TOP[kind] / w.sum()
    return out, bound


def check(got, want):
    out, bound = want
    got, = host(got)
    assert np.isfinite(got).all()
    off = np.abs(got.astype(np.float64) - out)
    assert (off <= bound).all(), float((off / np.maximum(bound, 1e-300)).max())
    assert (got[bound == 0] == 0).all()


def problem(rng, lens, Hq, Hkv, D, page, block, kind, spare=2):
    lens = np.array(lens, np.int32)
    pages = [-(-int(n) // page) for n in lens]
    P, W = sum(pages) + spare, max(max(pages), 1) + 1
    table = tables(rng, len(lens), W, page, P, pages)
    arrays = pools(rng, P, Hkv, page, D, block, kind)
    q = rng.standard_normal((len(lens), Hq, D)).astype(np.float32)
    return q, arrays, table, lens


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("lens,Hq,Hkv,D,page,block", [
    ([1], 1, 1, 1, 1, 1), ([0, 1, 2, 3], 2, 2, 7, 1, 1), ([5, 0, 17], 6, 2, 40, 2, 2), ([33, 64, 7], 4, 4, 64, 4, 2),
    ([31, 32, 33, 127, 128, 129], 8, 2, 128, 16, 16), ([63, 64, 65, 255, 256, 257], 12, 12, 64, 16, 4),
    ([100, 300, 511, 513], 16, 1, 128, 8, 8), ([40, 1], 17, 1, 128, 32, 1), ([200], 80, 2, 64, 64, 16),
    ([77, 150], 9, 3, 100, 16, 8), ([77, 150], 9, 3, 72, 16, 2), ([500, 3], 8, 8, 80, 128, 128), ([90], 14, 2, 33, 16, 16),
    ([700, 1200, 0, 1], 32, 8, 128, 64, 32), ([999], 14, 2, 64, 32, 16)])
def test_sizes(lens, Hq, Hkv, D, page, block, kind):
    rng = np.random.default_rng(D + page)
    note(f"decode8 {lens} {Hq}/{Hkv} {D} {page} {block} {kind}")
    q, arrays, table, lens = problem(rng, lens, Hq, Hkv, D, page, block, kind)
    c, *_ = cache_of(arrays, kind)
    check(cf.attention8_decode(dev(q), c, dev(table), dev(lens)), expected(q, arrays, kind, block, table, lens))


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("lens,Hq,Hkv,D,page,block", [([20001], 8, 2, 128, 64, 64), ([9000, 1, 4097], 6, 6, 64, 16, 16),
                                                      ([70000], 4, 1, 64, 128, 32)])
def test_long(lens, Hq, Hkv, D, page, block, kind):
    """Many parts of few sequences."""
    rng = np.random.default_rng(D)
    note(f"decode8 long {lens} {kind}")
    q, arrays, table, lens = problem(rng, lens, Hq, Hkv, D, page, block, kind)
    c, *_ = cache_of(arrays, kind)
    check(cf.attention8_decode(dev(q), c, dev(table), dev(lens)), expected(q, arrays, kind, block, table, lens))


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_large_batch(kind):
    rng = np.random.default_rng(5)
    note(f"decode8 batch {kind}")
    q, arrays, table, lens = problem(rng, rng.integers(0, 200, 150), 8, 4, 64, 16, 16, kind)
    c, *_ = cache_of(arrays, kind)
    check(cf.attention8_decode(dev(q), c, dev(table), dev(lens)), expected(q, arrays, kind, 16, table, lens))


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("layout", ["plain", "token_major", "odd", "padded"])
@pytest.mark.parametrize("D", [64, 128, 80])
def test_layouts(layout, D, kind):
    rng = np.random.default_rng(D)
    note(f"decode8 {layout} {D} {kind}")
    q, arrays, table, lens = problem(rng, [100, 33, 0], 8, 2, D, 16, 8, kind)
    c, *_ = cache_of(arrays, kind, layout)
    want = expected(q, arrays, kind, 8, table, lens)
    wide = np.full((3, 20), 77, np.int32)
    wide[:, 3:3 + table.shape[1]] = table
    t = dev(wide)[:, 3:3 + table.shape[1]]
    big = torch.full((4, 9, D + 3), 5.0, device="cuda")
    out = big[:3, :8, :D]
    check(cf.attention8_decode(placed(q, "padded" if layout != "odd" else "odd"), c, t, dev(lens), out=out), want)
    out.fill_(5.0)
    assert bool((big == 5.0).all())
    flat = torch.zeros(8, 3, D, device="cuda").transpose(0, 1)  # head-major
    check(cf.attention8_decode(dev(q.transpose(1, 0, 2)).transpose(0, 1), c, t, dev(lens), out=flat), want)


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 5.0])
def test_scale(scale, kind):
    rng = np.random.default_rng(1)
    note(f"decode8 scale {scale} {kind}")
    q, arrays, table, lens = problem(rng, [200, 17], 4, 2, 64, 16, 16, kind)
    c, *_ = cache_of(arrays, kind)
    check(cf.attention8_decode(dev(q), c, dev(table), dev(lens), scale=scale), expected(q, arrays, kind, 16, table, lens, scale))


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_magnitudes(kind):
    """q and the scales of K and V from very small to very large, next to each other."""
    rng = np.random.default_rng(2)
    for qs, kss, vss in ((1, 0, 60), (2.0 ** 60, -60, 0), (2.0 ** -60, 50, 100), (1, 0, 0), (2.0 ** 100, -105, 20),
                          (2.0 ** -120, 118, 0), (2.0 ** 115, -118, 10)):
        note(f"decode8 magnitudes {qs} {kss} {vss} {kind}")
        q, arrays, table, lens = problem(rng, [300, 40], 4, 2, 64, 16, 2, kind)
        q *= np.float32(qs)
        arrays[1] = (arrays[1] * np.float32(2.0 ** kss)).astype(np.float32)
        spread = rng.integers(-vss, 5, arrays[3].shape)
        arrays[3] = (arrays[3] * 2.0 ** spread).astype(np.float32)
        c, *_ = cache_of(arrays, kind)
        check(cf.attention8_decode(dev(q), c, dev(table), dev(lens)), expected(q, arrays, kind, 2, table, lens))


def test_a_large_scale_without_weight_costs_no_bits():
    """Two kinds of tokens: of weight 1 and scale 1, and of weight e^-80 and scale 2^60, side by side."""
    rng = np.random.default_rng(3)
    q, arrays, table, lens = problem(rng, [64], 1, 1, 64, 16, 1, "i8")
    q[:] = 1
    arrays[0][:] = np.uint8(1)
    far = np.arange(16) % 2 == 1
    arrays[1][:] = np.where(far, -1.25, 0.0)  # scores of 0 and -80
    arrays[3][:] = np.where(far, 2.0 ** 60, 1.0)
    c, *_ = cache_of(arrays, "i8")
    note("decode8 large scale")
    got, = host(cf.attention8_decode(dev(q), c, dev(table), dev(lens), scale=1.0))
    out, bound = expected(q, arrays, "i8", 1, table, lens, 1.0)
    assert (np.abs(got - out) <= bound).all()


@pytest.mark.parametrize("kind", ["i8", "e4m3"])
def test_what_no_row_sees_does_not_reach_it(kind):
    """NaN and infinite scales, and codes of no value, behind the last token and in pages of no sequence."""
    rng = np.random.default_rng(4)
    q, arrays, table, lens = problem(rng, [37, 5, 0, 64], 4, 2, 64, 16, 4, kind)
    want = expected(q, arrays, kind, 4, table, lens)
    for i in range(0, 4, 2):
        seen = np.zeros((len(arrays[i]), 16), bool)
        for b, n in enumerate(lens):
            for j in range(n):
                seen[table[b, j // 16], j % 16] = True
        arrays[i][~seen[:, None, :].repeat(2, 1)] = 0x7F if kind == "e4m3" else 0x80
        blocks = seen.reshape(-1, 4, 4).any(2)
        arrays[i + 1][~blocks[:, None, :].repeat(2, 1)] = rng.choice([np.nan, np.inf, -np.inf])
    table = np.where(table < 0, rng.choice([-1, 99999, -7], table.shape), table).astype(np.int32)
    c, *_ = cache_of(arrays, kind)
    note(f"decode8 unseen {kind}")
    check(cf.attention8_decode(dev(q), c, dev(table), dev(lens)), want)


def test_rows_that_are_no_numbers():
    """Bad pages, scales that are NaN, and q's NaN and infinities: those rows alone."""
    rng = np.random.default_rng(6)
    q, arrays, table, lens = problem(rng, [100, 100, 100, 100, 2000], 4, 2, 64, 16, 16, "i8")
    want, bound = expected(q, arrays, "i8", 16, table, lens)
    bad = np.zeros(q.shape[:2], bool)
    table[0, 3] = -1
    table[4, 100] = 1 << 30
    bad[[0, 4]] = True
    arrays[1][table[1, 2], 1] = np.nan  # K/V head 1: query heads 2 and 3
    arrays[3][table[2, 0], 0] = np.nan
    bad[1, 2:] = bad[2, :2] = True
    q[3, 1, 5], q[3, 2, 7] = np.nan, np.inf
    bad[3, 1:3] = True
    c, *_ = cache_of(arrays, "i8")
    note("decode8 bad rows")
    got, = host(cf.attention8_decode(dev(q), c, dev(table), dev(lens)))
    assert np.isnan(got[bad]).all()
    assert (np.abs(got[~bad] - want[~bad]) <= bound[~bad]).all()


def test_lengths_that_are_none():
    rng = np.random.default_rng(7)
    q, arrays, table, lens = problem(rng, [48, 48, 48], 2, 1, 64, 16, 16, "i8", spare=3)
    table[:, 3] = np.setdiff1d(np.arange(12), table[:, :3].ravel())[:3]  # the table is full: four pages
    c, *_ = cache_of(arrays, "i8")
    note("decode8 lengths")
    odd = np.array([-5, 1 << 30, 48], np.int32)
    want = expected(q, arrays, "i8", 16, table, np.array([0, 64, 48]))
    check(cf.attention8_decode(dev(q), c, dev(table), dev(odd)), want)
    # No pages, no table: 0, or NaN where a sequence has tokens.
    none = cf.Cache8.empty(0, 1, 16, 64)
    got, = host(cf.attention8_decode(dev(q), none, dev(table), dev(np.array([0, 3, -1], np.int32))))
    assert (got[[0, 2]] == 0).all() and np.isnan(got[1]).all()
    got, = host(cf.attention8_decode(dev(q), c, dev(table[:, :0]), dev(lens)))
    assert (got == 0).all()


def test_as_the_cache_is_written():
    """Tokens written one by one and all at once, read back, and attended to: the values read back are those attended to."""
    rng = np.random.default_rng(8)
    page, H, D, n = 16, 2, 64, 50
    for dtype in (torch.int8, torch.float8_e4m3fn):
        c = cf.Cache8.empty(8, H, page, D, block=8, dtype=dtype)
        table = dev(np.array([[3, 1, 7, 5]], np.int32))
        lens, cu = dev(np.array([0], np.int32)), dev(np.array([0, n - 5], np.int32))
        k, v = (dev(rng.standard_normal((n, H, D)).astype(np.float32)) for _ in range(2))
        note(f"decode8 as written {dtype}")
        lens = cf.cache8_append(k[:n - 5], v[:n - 5], cu, c, table, lens)
        one = dev(np.array([0, 1], np.int32))
        for i in range(n - 5, n):
            lens = cf.cache8_append(k[i:i + 1], v[i:i + 1], one, c, table, lens)
        assert int(lens) == n
        kk, vv = cf.cache8_read(c, table, dev(np.array([0, n], np.int32)), n)
        # The block's largest over 127 (i8: less than a step of it), or 2^-4 of the value (floats).
        step = 2 * k.abs().max() / 127 if dtype == torch.int8 else k.abs().max() * 2.0 ** -4
        assert float((kk - k).abs().max()) <= float(step)
        q = rng.standard_normal((1, 6, D)).astype(np.float32)
        kh, vh = host(kk, vv)
        out = np.zeros((1, 6, D))
        for h in range(6):
            o, _ = paged.attend(q[0, h:h + 1], kh[:, h // 3], vh[:, h // 3], [n], D ** -0.5)
            out[0, h] = o[0]
        got, = host(cf.attention8_decode(dev(q), c, table, lens))
        # kk, vv are rounded to FP32 (2^-24 each), the rest as the bound of the same sums.
        assert np.abs(got - out).max() <= 2.0 ** -24 * 400 * np.abs(vh).max()


def test_streams_threads_and_graphs():
    """On another stream, with a workspace full of NaN, and captured twice with workspaces of their own: each replay is
    the eager call's result, bit for bit."""
    rng = np.random.default_rng(9)
    q, arrays, table, lens = problem(rng, [3000, 10, 700], 8, 2, 128, 16, 16, "i8")
    c, *parts = cache_of(arrays, "i8")
    t, n = dev(table), dev(lens)
    qd = dev(q)
    note("decode8 streams")
    want = cf.attention8_decode(qd, c, t, n)
    need = cf.cfp32_attention8_decode_workspace_bytes(3, 8, 2, 128, table.shape[1], 16)
    assert need > 0
    ws = cf.Workspace()
    ws.get(need, qd.device).view(torch.float32 if need % 4 == 0 else torch.uint8).fill_(float("nan"))
    assert torch.equal(cf.attention8_decode(qd, c, t, n, workspace=ws), want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = cf.attention8_decode(qd, c, t, n, stream=st)
    st.synchronize()
    assert torch.equal(got, want)
    graphs, outs, spaces = [], [], []
    torch.cuda.synchronize()
    for _ in range(2):
        g, w = torch.cuda.CUDAGraph(), cf.Workspace()
        w.get(need, qd.device)
        with torch.cuda.stream(st):
            with torch.cuda.graph(g, stream=st):
                outs.append(cf.attention8_decode(qd, c, t, n, workspace=w, stream=st))
        graphs.append(g)
        spaces.append(w)
    for i in range(3):
        qd.copy_(torch.randn_like(qd))
        n.copy_(dev(np.array([2999 - i, i, 700], np.int32)))
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = cf.attention8_decode(qd, c, t, n)
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_pools_beyond_32_bits():
    stride = (1 << 31) + 64
    rng = np.random.default_rng(10)
    q, arrays, table, lens = problem(rng, [30], 2, 1, 64, 16, 8, "i8", spare=0)
    note("decode8 large strides")
    want = expected(q, arrays, "i8", 8, table, lens)
    base = torch.zeros(stride + 16 * 64, dtype=torch.int8, device="cuda")
    k = base.as_strided((2, 1, 16, 64), (stride, 16 * 64, 64, 1))
    k.copy_(dev(arrays[0]).view(torch.int8))
    c = cf.Cache8(k, dev(arrays[2]).view(torch.int8), dev(arrays[1]), dev(arrays[3]))
    check(cf.attention8_decode(dev(q), c, dev(table), dev(lens)), want)


def test_the_helper_refuses():
    c = cf.Cache8.empty(3, 2, 16, 64)
    t, n = torch.zeros(2, 3, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    q = torch.zeros(2, 4, 64, device="cuda")
    for bad in ((q[:, :3], c, t, n), (q[..., :32], c, t, n), (q, c, t[:1], n), (q, c, t, n[:1])):
        with pytest.raises(ValueError):
            cf.attention8_decode(*bad)
    for bad in ((q.half(), c, t, n), (q, c, t.long(), n), (q.cpu(), c, t, n), (q, None, t, n)):
        with pytest.raises(TypeError):
            cf.attention8_decode(*bad)
    with pytest.raises(ValueError):
        cf.attention8_decode(q, c, t, n, out=torch.zeros(2, 4, 32, device="cuda"))
    with pytest.raises(cf.Cfp32Error):
        cf.attention8_decode(q, c, t, n, scale=float("inf"))
