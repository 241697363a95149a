"""GPU tests of the rotary call against its formulas in 64 bits (angles in 80).

With e = 2^-24 and a pair (u, v): sine and cosine are each off by at most 2.5 e
(the reduced angle's rounding, and those of a polynomial), the amplitude and its
product by e each, the two products and the sum by another 2 e: together less
than 8 e a (|u| + |v|).  The angle is off by 4 x 2^-53 of itself (the frequency,
its conversion to turns, the product).  FP16 results are off by half a step more:
2^-11 of the value, 2^-25 among subnormals.
"""
import numpy as np
import pytest
import torch

import compensated_fp32_projection_amd as cf
from gpu_helpers import note

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


def oracle(x, f, pos, layout, amplitude, transpose, f16):
    """(y, bound) of x [T, H, D], numpy FP32 or FP16."""
    x = x.astype(np.float64)
    n = len(f)
    angle = pos.astype(np.longdouble)[:, None] * f.astype(np.longdouble)
    c, s = (t.astype(np.float64)[:, None, :] for t in (np.cos(angle), np.sin(angle)))
    if transpose:
        s = -s
    first = np.arange(n) * (1 if layout == "half" else 2)
    second = first + (n if layout == "half" else 1)
    y, bound = x.copy(), np.zeros_like(x)
    u, v = x[..., first], x[..., second]
    y[..., first] = amplitude * (u * c - v * s)
    y[..., second] = amplitude * (v * c + u * s)
    b = (8 * E + 4 * 2.0 ** -53 * np.abs(angle.astype(np.float64))[:, None, :]) * abs(amplitude) * (np.abs(u) + np.abs(v))
    bound[..., first] = bound[..., second] = b + 2.0 ** -149
    if f16:
        bound = np.where(bound > 0, bound * (1 + 2.0 ** -10) + np.abs(y) * 2.0 ** -11 + 2.0 ** -25, 0)
    return y, bound


def check(got, x, f, pos, layout="half", amplitude=1.0, transpose=False):
    y, bound = oracle(x.cpu().numpy(), f.cpu().numpy(), pos, layout, amplitude, transpose, x.dtype == torch.float16)
    off = np.abs(got.cpu().numpy().astype(np.float64) - y)
    assert (off <= bound).all(), (float((off / np.maximum(bound, 1e-300)).max()))


def placed(x, how):
    if how == "head_major":
        return x.transpose(0, 1).contiguous().transpose(0, 1)
    if how == "odd":
        return torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")[1:].view(x.shape).copy_(x)
    if how == "padded":
        T, H, D = x.shape
        return torch.zeros(T + 1, H + 1, D + 3, dtype=x.dtype, device="cuda")[:T, :H, :D].copy_(x)
    return x


def inputs(T, Hq, Hkv, D, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(T, h, D, generator=g, device="cuda").to(dtype) for h in (Hq, Hkv)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,R", [(2, 2), (6, 4), (40, 20), (64, 64), (64, 16), (80, 80), (128, 128), (130, 130), (128, 2),
                                 (1024, 1024), (65, 32), (96, 0)])
def test_sizes(D, R, layout, dtype):
    for T, Hq, Hkv in ((1, 1, 0), (3, 4, 2), (37, 9, 3)):
        note(f"rotary {T} {Hq}/{Hkv} {D} {R} {layout} {dtype}")
        q, k = inputs(T, Hq, Hkv, D, dtype, T + D)
        f = cf.rotary_frequencies(R)[0] if R else torch.empty(0, dtype=torch.float64, device="cuda")
        pos = np.random.default_rng(T).integers(0, 10000, T)
        for transpose in (False, True):
            yq, yk = cf.rotary(q, k if Hkv else None, f, torch.from_numpy(pos).cuda(), layout=layout, transpose=transpose)
            check(yq, q, f, pos, layout, 1.0, transpose)
            if Hkv:
                check(yk, k, f, pos, layout, 1.0, transpose)
            else:
                assert yk is None


@pytest.mark.parametrize("T,Hq,Hkv,D", [(700, 32, 8, 128), (1025, 14, 2, 64), (3001, 2, 1, 128)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_many_tokens(T, Hq, Hkv, D, dtype):
    q, k = inputs(T, Hq, Hkv, D, dtype)
    f, a = cf.rotary_frequencies(D, scaling="parts", factor=8.0, trained=4096)
    yq, yk = cf.rotary(q, k, f, amplitude=a)
    check(yq, q, f, np.arange(T), amplitude=a)
    check(yk, k, f, np.arange(T), amplitude=a)


@pytest.mark.parametrize("how", ["head_major", "odd", "padded"])
@pytest.mark.parametrize("out", ["new", "same", "in_place"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
def test_strides(how, out, dtype):
    q, k = inputs(19, 6, 2, 64, dtype)
    f = cf.rotary_frequencies(32)[0]
    pos = np.arange(19) * 7
    qq, kk = placed(q, how), placed(k, how)
    kw = {}
    if out == "same":
        kw = dict(q_out=placed(torch.zeros_like(q), how), k_out=placed(torch.zeros_like(k), how))
    if out == "in_place":
        kw = dict(q_out=qq, k_out=kk)
    yq, yk = cf.rotary(qq, kk, f, torch.from_numpy(pos).cuda(), layout="interleaved", **kw)
    check(yq, q, f, pos, "interleaved")
    check(yk, k, f, pos, "interleaved")
    if out != "in_place":
        assert torch.equal(qq, q) and torch.equal(kk, k)


def test_rows_beside_the_outputs_are_left():
    q, k = inputs(5, 3, 1, 40, torch.float32)
    f = cf.rotary_frequencies(20)[0]
    big = torch.full((7, 5, 44), 7.0, device="cuda")
    cf.rotary(q, None, f, q_out=big[1:6, 1:4, 2:42])
    check(big[1:6, 1:4, 2:42], q, f, np.arange(5))
    big[1:6, 1:4, 2:42] = 7.0
    assert bool((big == 7.0).all())


def test_broadcast_inputs():
    """Stride 0: one row for all tokens, or one head for all."""
    x, _ = inputs(1, 4, 1, 64, torch.float32)
    f = cf.rotary_frequencies(64)[0]
    wide = x.expand(9, 4, 64)
    check(cf.rotary(wide, None, f)[0], wide.contiguous(), f, np.arange(9))
    one = inputs(9, 1, 1, 64, torch.float32)[0].expand(9, 3, 64)
    check(cf.rotary(one, None, f)[0], one.contiguous(), f, np.arange(9))
    with pytest.raises(cf.Cfp32Error):
        cf.rotary(wide, None, f, q_out=torch.zeros(1, 4, 64, device="cuda").expand(9, 4, 64))


@pytest.mark.parametrize("pos", [[0, -1, -1000, 5], [2 ** 20, 2 ** 20 + 1, 2 ** 24 + 3, 2 ** 31 - 1],
                                 [2 ** 31, 2 ** 33 + 7, 123456789012, -2 ** 33]])
def test_far_and_negative_positions(pos):
    q, k = inputs(4, 4, 2, 128, torch.float32)
    f = cf.rotary_frequencies(128)[0]
    p = np.array(pos, np.int64)
    yq, yk = cf.rotary(q, k, f, torch.from_numpy(p).cuda())
    check(yq, q, f, p)
    check(yk, k, f, p)


def test_every_angle_of_a_turn():
    """A pair (1, 0) at all angles: cosine and sine themselves, each quarter and the borders between them."""
    T = 4096
    q = torch.zeros(T, 1, 2, device="cuda")
    q[..., 0] = 1.0
    for turn in (2 * np.pi / T, 2 * np.pi / 8, np.pi / 2, 1.0):
        f = torch.tensor([turn], dtype=torch.float64, device="cuda")
        check(cf.rotary(q, None, f)[0], q, f, np.arange(T))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_transpose_is_the_gradient(layout):
    """<g, R x> = <R' g, x>, and differences along a direction: the map is linear."""
    x, _ = inputs(11, 5, 1, 64, torch.float32, 1)
    g, _ = inputs(11, 5, 1, 64, torch.float32, 2)
    f, a = cf.rotary_frequencies(48, scaling="parts", factor=4.0, trained=100)
    y = cf.rotary(x, None, f, layout=layout, amplitude=a)[0]
    gx = cf.rotary(g, None, f, layout=layout, amplitude=a, transpose=True)[0]
    left, right = (g.double() * y.double()).sum(), (gx.double() * x.double()).sum()
    room = 16 * E * a * (g.double().abs().sum() * x.abs().max() + x.double().abs().sum() * g.abs().max())
    assert abs(float(left - right)) <= float(room)
    d, _ = inputs(11, 5, 1, 64, torch.float32, 3)
    # h a power of two: the errors of two outputs (16 e a max) and of x + h d (2 e a max) over h, and the gradient's own.
    h = 2.0 ** -3
    moved = cf.rotary(x + h * d, None, f, layout=layout, amplitude=a)[0]
    lost = 40 * E * a * float(x.abs().max() + d.abs().max()) / h * float(g.double().abs().sum())
    lost += 16 * E * a * float(g.abs().max() * d.double().abs().sum())
    want = (gx.double() * d.double()).sum()
    got = (g.double() * (moved.double() - y.double())).sum() / h
    assert abs(float(got - want)) <= lost


def test_special_values_stay_in_their_pairs():
    q, _ = inputs(3, 2, 1, 8, torch.float32)
    q[1, 0, 2] = float("nan")
    q[1, 1, 0] = float("inf")
    f = cf.rotary_frequencies(8)[0]
    y = cf.rotary(q, None, f)[0].cpu()
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[1, 0, [2, 6]] = True
    want[1, 1, [0, 4]] = True
    assert torch.equal(bad, want)


def test_another_stream_and_a_graph():
    q, k = inputs(33, 4, 2, 64, torch.float32)
    f = cf.rotary_frequencies(64)[0]
    pos = torch.arange(33, device="cuda")
    want = cf.rotary(q, k, f, pos)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = cf.rotary(q, k, f, pos, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    yq, yk = torch.empty_like(q), torch.empty_like(k)
    with torch.cuda.graph(g):
        cf.rotary(q, k, f, pos, q_out=yq, k_out=yk)
    for i in range(3):
        pos.add_(i)
        q.mul_(0.5)
        g.replay()
        torch.cuda.synchronize()
        want = cf.rotary(q, k, f, pos)
        assert torch.equal(yq, want[0]) and torch.equal(yk, want[1])
