"""Rotary frequencies (host only) against their formulas, and the refusals of the
rotary calls: no kernel is launched."""
import ctypes
import math

import pytest
import torch

import compensated_fp32_projection_amd as cf

FAKE, FAKE2 = 1 << 20, 1 << 21  # never dereferenced
E, OK = cf.ERR_INVALID_VALUE, cf.OK


def frequencies(R, **kw):
    f, a = cf.rotary_frequencies(R, device="cpu", **kw)
    assert f.dtype == torch.float64 and f.shape == (R // 2,)
    return f.tolist(), a


# Two roundings of pow's argument of up to 10 and its own last bits: 2^-48 covers them.
def close(got, want):
    return all(abs(a - b) <= 2.0 ** -48 * abs(b) for a, b in zip(got, want))


@pytest.mark.parametrize("R", [2, 4, 20, 64, 128, 1024])
@pytest.mark.parametrize("theta", [10000.0, 500000.0, 1.0])
def test_frequencies(R, theta):
    plain = [theta ** (-2 * i / R) for i in range(R // 2)]
    f, a = frequencies(R, theta=theta)
    assert close(f, plain) and a == 1.0
    f, a = frequencies(R, theta=theta, scaling="linear", factor=4.0)
    assert close(f, [x / 4 for x in plain]) and a == 1.0
    f, a = frequencies(R, theta=theta, scaling="ntk", factor=8.0)
    base = theta * 8.0 ** (R / (R - 2)) if R > 2 else theta
    assert close(f, [base ** (-2 * i / R) for i in range(R // 2)]) and a == 1.0
    if R > 2:  # the fastest pair is left, the slowest interpolated
        assert f[0] == 1.0 and abs(f[-1] * 8.0 / plain[-1] - 1) < 1e-12
    f, a = frequencies(R, theta=theta, scaling="parts", factor=16.0, trained=2048, slow=1, fast=32)
    assert abs(a - (1 + 0.1 * math.log(16))) < 1e-15
    for x, y in zip(f, plain):
        turns = 2048 * y / (2 * math.pi)
        g = min(max((turns - 1) / 31, 0.0), 1.0)
        assert abs(x - (g * y + (1 - g) * y / 16)) <= 2.0 ** -46 * y


def test_refused_frequencies():
    good = dict(theta=10000.0, rotary_dim=64, scaling="parts", factor=2.0, trained=100.0, slow=1.0, fast=32.0, device="cpu")
    cf.rotary_frequencies(**good)
    nan, inf = float("nan"), float("inf")
    for bad in (dict(theta=0.0), dict(theta=-1.0), dict(theta=nan), dict(theta=inf), dict(rotary_dim=0), dict(rotary_dim=3),
                dict(rotary_dim=-2), dict(rotary_dim=1026), dict(factor=0.5), dict(factor=nan), dict(factor=inf),
                dict(trained=0.0), dict(trained=inf), dict(slow=32.0), dict(slow=nan), dict(fast=inf),
                dict(scaling="ntk", theta=1e300, factor=1e300, rotary_dim=4)):
        with pytest.raises(cf.Cfp32Error):
            cf.rotary_frequencies(**{**good, **bad})
    with pytest.raises(ValueError):
        cf.rotary_frequencies(64, scaling="other")
    out = (ctypes.c_double * 32)()
    assert cf.cfp32_rotary_frequencies(1e4, 64, 4, 2.0, 1.0, 1.0, 2.0, out, out) == E
    assert cf.cfp32_rotary_frequencies(1e4, 64, -1, 2.0, 1.0, 1.0, 2.0, out, out) == E
    assert cf.cfp32_rotary_frequencies(1e4, 64, 0, 2.0, 1.0, 1.0, 2.0, None, out) == E
    assert cf.cfp32_rotary_frequencies(1e4, 64, 0, 2.0, 1.0, 1.0, 2.0, out, None) == E


CALL = dict(q=FAKE, q_tok=128, q_head=64, k=FAKE, k_tok=64, k_head=64, type=0, positions=FAKE, frequencies=FAKE, amplitude=1.0,
            layout=0, transpose=0, q_out=FAKE2, qo_tok=128, qo_head=64, k_out=FAKE2, ko_tok=64, ko_head=64, T=5, Hq=2, Hkv=1,
            D=64, R=64, stream=None)


def call(**changed):
    assert set(changed) <= set(CALL)
    return cf.cfp32_rotary(**{**CALL, **changed})


def test_the_call_as_it_stands_is_accepted():
    if torch.cuda.is_available():
        pytest.skip("would run on made-up pointers")
    assert call() == cf.ERR_UNSUPPORTED_DEVICE
    assert call(k=None, k_out=None, Hkv=0) == cf.ERR_UNSUPPORTED_DEVICE
    assert call(q_out=FAKE, k_out=FAKE) == cf.ERR_UNSUPPORTED_DEVICE  # in place
    assert call(positions=None, R=0, frequencies=None) == cf.ERR_UNSUPPORTED_DEVICE


@pytest.mark.parametrize("changed", [
    dict(q=None), dict(k=None), dict(q_out=None), dict(k_out=None), dict(frequencies=None), dict(frequencies=FAKE + 4),
    dict(positions=FAKE + 4), dict(q=FAKE + 2), dict(k_out=FAKE2 + 2), dict(type=1, q=FAKE + 1), dict(type=2), dict(type=-1),
    dict(layout=2), dict(layout=-1), dict(T=-1), dict(T=1 << 31), dict(Hq=-1), dict(Hkv=-1), dict(D=1025), dict(D=-1),
    dict(R=66), dict(R=63), dict(R=-2), dict(q_tok=-1), dict(q_head=-64), dict(qo_tok=64), dict(ko_tok=63), dict(qo_head=32),
    dict(ko_tok=0), dict(q_tok=1 << 47), dict(amplitude=float("nan")), dict(amplitude=1e39),
    dict(q_out=FAKE, qo_tok=256), dict(Hq=1 << 21, qo_tok=1 << 30)])
def test_refusals(changed):
    assert call(**changed) == E


def test_empty_problems_are_no_ops():
    assert call(T=0, q=None, k=None, q_out=None, k_out=None) == OK
    assert call(Hq=0, Hkv=0) == OK
    assert call(D=0, R=0) == OK


def test_the_helper_checks_its_tensors():
    q, f = torch.zeros(4, 2, 64), torch.zeros(32, dtype=torch.float64)
    with pytest.raises(TypeError):
        cf.rotary(q, q, f)
    with pytest.raises(ValueError):
        cf.rotary(q, q, f, layout="other")
