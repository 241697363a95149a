"""GPU tests of cfp32_attention_prompt against the definition in FP64 (tolerance
derived in attention_reference.py): sequence lengths around every tile edge,
empty sequences and rows that see no key, head sizes and groups, strides and
alignment, what masked places hold, ranges FP16 does not reach, streams and
graphs."""
import numpy as np
import pytest
import torch

import attention_reference as ref
import compensated_fp32_projection_amd as cf
from gpu_helpers import note

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16}


def starts(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def make(seed, lq, lk, Hq, Hkv, D, kv):
    rng = np.random.default_rng(seed)
    q = rng.standard_normal((sum(lq), Hq, D), dtype=np.float32) * 1.5
    k = rng.standard_normal((sum(lk), Hkv, D), dtype=np.float32) * 1.5
    v = rng.standard_normal((sum(lk), Hkv, D), dtype=np.float32)
    if kv == "f16":
        k, v = k.astype(np.float16), v.astype(np.float16)
    return q, k, v


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def call(q, k, v, cu_q, cu_k, **kw):
    o = cf.attention_prompt(q, k, v, dev(cu_q), dev(cu_k), **kw)
    torch.cuda.synchronize()
    return o.cpu().numpy()


def check(got, want, bound, what=""):
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    err = np.abs(got.astype(np.float64) - want)
    worst = np.max(err - bound)
    assert worst <= 0, f"{what}: off by {err.max():.3g}, {worst:.3g} over the bound"
    assert (got[bound == 0] == 0).all(), f"{what}: rows that see nothing"


LENS = [
    ([1], [1]), ([37], [37]), ([63, 64, 65], [63, 64, 65]), ([127, 128, 129], [127, 128, 129]), ([300], [300]),
    ([1, 0, 5, 0, 0, 200, 1], [1, 0, 5, 0, 0, 200, 1]),   # empty sequences
    ([1, 2, 33, 100], [70, 64, 191, 600]),                # rows that go on from a cached prefix
    ([40, 7, 130], [10, 0, 128]),                         # causal rows that see nothing
    ([1] * 70, list(range(1, 71))),                       # more sequences than lanes
]


@pytest.mark.parametrize("kv", ["f32", "f16"])
@pytest.mark.parametrize("lens", LENS, ids=lambda x: "-".join(map(str, x[0][:7])))
@pytest.mark.parametrize("causal", [True, False])
def test_lengths(lens, kv, causal):
    lq, lk = lens
    note(f"prompt lengths {lq} {lk} {kv} causal={causal}")
    q, k, v = make(len(lq) + sum(lk), lq, lk, 4, 2, 64, kv)
    cu_q, cu_k = starts(lq), starts(lk)
    got = call(dev(q), dev(k), dev(v), cu_q, cu_k, causal=causal)
    want, bound, _ = ref.prompt(q, k, v, cu_q, cu_k, causal)
    check(got, want, bound)


@pytest.mark.parametrize("kv", ["f32", "f16"])
@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 1), (2, 1, 2), (3, 3, 10), (9, 3, 40), (5, 1, 63), (14, 2, 64), (8, 8, 80),
                                      (6, 2, 96), (4, 1, 127), (32, 8, 128)])
def test_heads(Hq, Hkv, D, kv):
    note(f"prompt heads {Hq}/{Hkv} x {D} {kv}")
    lq, lk = [70, 150], [90, 150]
    q, k, v = make(Hq * D, lq, lk, Hq, Hkv, D, kv)
    cu_q, cu_k = starts(lq), starts(lk)
    want, bound, _ = ref.prompt(q, k, v, cu_q, cu_k)
    check(call(dev(q), dev(k), dev(v), cu_q, cu_k), want, bound)


@pytest.mark.parametrize("kv", ["f32", "f16"])
@pytest.mark.parametrize("D", [64, 128, 48])
@pytest.mark.parametrize("layout", ["head_major", "odd_offset", "padded_rows", "one_head_for_all", "packed_qkv"])
def test_layouts(layout, D, kv):
    note(f"prompt layout {layout} D={D} {kv}")
    T, Hq, Hkv = 140, 4, 2
    q, k, v = make(T + D, [T], [T], Hq, Hkv, D, kv)
    tq, tk, tv = dev(q), dev(k), dev(v)
    out = None
    if layout == "head_major":
        tq, tk, tv = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (tq, tk, tv))
        out = torch.full((Hq, T, D), 7.0, device="cuda").transpose(0, 1)
    elif layout == "odd_offset":  # one element past the allocation: no wide loads
        def off(x):
            y = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(x.shape)
            return y.copy_(x)
        tq, tk, tv, out = off(tq), off(tk), off(tv), off(torch.full((T, Hq, D), 7.0, device="cuda"))
    elif layout == "padded_rows":
        def pad(x):
            y = torch.full((x.shape[0], x.shape[1] + 1, D + 3), float("nan"), dtype=x.dtype, device="cuda")
            y[:, :x.shape[1], :D] = x
            return y[:, :x.shape[1], :D]
        tq, tk, tv, out = pad(tq), pad(tk), pad(tv), pad(torch.full((T, Hq, D), 7.0, device="cuda"))
    elif layout == "one_head_for_all":
        tk, tv = tk[:, :1].expand(T, Hkv, D), tv[:, :1].expand(T, Hkv, D)
        k, v = np.repeat(k[:, :1], Hkv, 1), np.repeat(v[:, :1], Hkv, 1)
    else:
        tk = torch.cat([tk, tv], dim=1)
        tk, tv = tk[:, :Hkv], tk[:, Hkv:]
    cu = starts([T])
    want, bound, _ = ref.prompt(q, k, v, cu, cu)
    check(call(tq, tk, tv, cu, cu, out=out), want, bound, layout)


@pytest.mark.parametrize("kv", ["f32", "f16"])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_what_is_masked_does_not_matter(kv, bad):
    """Non-finite K and V of other sequences, of tokens outside all sequences
    and of later tokens leave a row alone; a row that sees one shows it."""
    note(f"prompt masked {bad} {kv}")
    Hq, Hkv, D = 4, 2, 64
    lens, at = [5, 100, 150, 30], 90   # token 90 of the third sequence is bad
    q, k, v = make(3, [3] + lens + [9], [3] + lens + [9], Hq, Hkv, D, kv)
    cu = starts([3] + lens + [9])[1:-1]
    want, bound, written = ref.prompt(q, k, v, cu, cu)
    for x in (k, v):
        x[:3] = bad
        x[-9:] = bad
        x[cu[0]:cu[1]] = bad
    if np.isnan(bad):
        k[cu[2] + at] = bad
    v[cu[2] + at, :, 7] = bad
    out = torch.full((q.shape[0], Hq, D), 7.0, device="cuda")
    got = call(dev(q), dev(k), dev(v), cu, cu, out=out)
    assert (got[~written] == 7.0).all()
    assert not np.isfinite(got[cu[0]:cu[1]]).any()
    seen = slice(cu[2] + at, cu[3])
    if np.isnan(bad):
        assert np.isnan(got[seen]).all()
    else:
        assert (got[seen, :, 7] == bad).all()
        keep = np.arange(D) != 7
        check(got[seen][..., keep], want[seen][..., keep], bound[seen][..., keep], "beside it")
    rest = np.r_[cu[1]:cu[2] + at, cu[3]:cu[4]]
    check(got[rest], want[rest], bound[rest], "rows that do not see it")


def test_opposite_infinities_give_nan():
    q, k, v = make(4, [80], [80], 2, 1, 64, "f32")
    v[10, 0, 3], v[70, 0, 3] = np.inf, -np.inf
    cu = starts([80])
    note("prompt opposite infinities")
    got = call(dev(q), dev(k), dev(v), cu, cu)
    assert np.isfinite(got[:10]).all()
    assert (got[10:70, :, 3] == np.inf).all() and np.isnan(got[70:, :, 3]).all()


@pytest.mark.parametrize("sq,sk,sv", [(1e-20, 1e20, 1.0), (1e18, 1e-18, 1e30), (1.0, 1.0, 1e-30), (3e4, 1e-5, 7e4)])
def test_ranges_of_fp32(sq, sk, sv):
    """Magnitudes far outside FP16's: the parts are taken at the operands' own scale."""
    note(f"prompt ranges {sq} {sk} {sv}")
    q, k, v = make(5, [130], [130], 2, 2, 64, "f32")
    q, k, v = (x * np.float32(f) for x, f in ((q, sq), (k, sk), (v, sv)))
    cu = starts([130])
    want, bound, _ = ref.prompt(q, k, v, cu, cu)
    check(call(dev(q), dev(k), dev(v), cu, cu), want, bound)


def test_values_of_very_different_tiles():
    """A sequence whose value magnitudes change by powers of 2^20 from one 64
    keys to the next: FP32-grade relative to what each row sums, also in rows
    that see only the small ones."""
    rng = np.random.default_rng(6)
    T, D = 256, 64
    q, k, v = make(6, [T], [T], 1, 1, D, "f32")
    v *= np.float32(2.0) ** (20 * rng.integers(-2, 3, T // 64)).repeat(64)[:, None, None].astype(np.float32)
    cu = starts([T])
    note("prompt tiles of different magnitude")
    want, bound, _ = ref.prompt(q, k, v, cu, cu)
    check(call(dev(q), dev(k), dev(v), cu, cu), want, bound)


@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 3.0])
def test_scale(scale):
    """0 averages, a negative scale turns the order round, a large one makes the softmax one-hot."""
    note(f"prompt scale {scale}")
    q, k, v = make(7, [100], [100], 2, 1, 64, "f32")
    cu = starts([100])
    want, bound, _ = ref.prompt(q, k, v, cu, cu, scale=scale)
    check(call(dev(q), dev(k), dev(v), cu, cu, scale=scale), want, bound)


def test_zero_inputs():
    q, k, v = make(8, [66], [66], 2, 1, 64, "f32")
    cu = starts([66])
    note("prompt zeros")
    got = call(dev(q * 0), dev(k * 0), dev(v), cu, cu)
    want, bound, _ = ref.prompt(q * 0, k * 0, v, cu, cu)
    check(got, want, bound)
    assert (call(dev(q), dev(k), dev(v * 0), cu, cu) == 0).all()


@pytest.mark.parametrize("kv", ["f32", "f16"])
def test_offsets_beyond_32_bits(kv):
    """Token strides that put the last rows more than 2^32 bytes from the first."""
    T, D, stride = 140, 64, (1 << 24) + 8
    if kv == "f32":
        stride //= 2
    q, k, v = make(9, [T], [T], 1, 1, D, kv)
    note(f"prompt large offsets {kv}")
    def far(x):
        y = torch.empty((T - 1) * stride + D, dtype=DT[kv], device="cuda").as_strided((T, 1, D), (stride, D, 1))
        return y.copy_(dev(x))
    cu = starts([T])
    want, bound, _ = ref.prompt(q, k, v, cu, cu)
    check(call(dev(q), far(k), far(v), cu, cu), want, bound)


def test_repeats_and_other_stream():
    """The same bits every time; on a side stream with its own workspace."""
    q, k, v = make(10, [200, 77], [200, 90], 8, 2, 128, "f32")
    cu_q, cu_k = dev(starts([200, 77])), dev(starts([200, 90]))
    tq, tk, tv = dev(q), dev(k), dev(v)
    a = cf.attention_prompt(tq, tk, tv, cu_q, cu_k)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    b = cf.attention_prompt(tq, tk, tv, cu_q, cu_k, stream=side, workspace=cf.Workspace())
    c = cf.attention_prompt(tq, tk, tv, cu_q, cu_k)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("kv", ["f32", "f16"])
def test_graph_replays(kv):
    """Captured once, replayed on new inputs and new sequence offsets."""
    q, k, v = make(11, [150, 60], [150, 60], 4, 2, 64, kv)
    tq, tk, tv, cu = dev(q), dev(k), dev(v), dev(starts([150, 60]))
    out, ws = torch.empty_like(tq), cf.Workspace()
    note(f"prompt graph {kv}")
    cf.attention_prompt(tq, tk, tv, cu, out=out, workspace=ws)
    torch.cuda.synchronize()
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(st):
        with torch.cuda.graph(g, stream=st):
            cf.attention_prompt(tq, tk, tv, cu, out=out, workspace=ws, stream=st)
    torch.cuda.synchronize()
    for r in range(4):
        tq.copy_(torch.randn_like(tq))
        cu.copy_(dev(starts([20 + 50 * r, 190 - 50 * r])))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, cf.attention_prompt(tq, tk, tv, cu, workspace=cf.Workspace())), f"replay {r}"
