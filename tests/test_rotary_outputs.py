"""The rotary call's outputs, on the host: its own input or memory of its own, never the other's."""
import os

import pytest
import torch

import compensated_fp32_projection_amd as cf

A, B, C, D = (i << 20 for i in range(1, 5))  # never dereferenced
OK = cf.ERR_UNSUPPORTED_DEVICE


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(cf.LIB_PATH):
        from compensated_fp32_projection_amd import build
        build.build()
    return cf.load_library()


def call(q, k, q_out, k_out, Hq=2, Hkv=2):
    return cf.cfp32_rotary(q, 128, 64, k, 128, 64, 0, None, A, 1.0, 0, 0, q_out, 128, 64, k_out, 128, 64, 5, Hq, Hkv, 64, 64, None)


def test_outputs():
    if torch.cuda.is_available():
        pytest.skip("would run on made-up pointers")
    assert call(A, B, C, D) == call(A, B, A, B) == call(A, B, A, D) == call(A, B, C, B) == call(A, A, C, D) == OK
    for bad in ((A, B, C, C), (A, B, B, A), (A, B, B, D), (A, B, C, A), (A, B, A, A), (A, B, B, B)):
        assert call(*bad) == cf.ERR_INVALID_VALUE, bad
    # Without heads nothing is read or written.
    assert call(A, B, C, C, Hkv=0) == call(A, None, A, None, Hkv=0) == call(A, B, B, A, Hq=0) == OK


@pytest.mark.gpu
def test_the_helper():
    q, k = torch.randn(5, 2, 64, device="cuda"), torch.randn(5, 2, 64, device="cuda")
    f, one = cf.rotary_frequencies(64)[0], torch.empty(5, 2, 64, device="cuda")
    want = q.clone(), k.clone()
    for kw in (dict(q_out=k, k_out=q), dict(q_out=k), dict(k_out=q), dict(q_out=one, k_out=one), dict(q_out=q, k_out=q)):
        for stream in (None, torch.cuda.current_stream()):  # the native form, and not
            with pytest.raises(ValueError, match="in this order"):
                cf.rotary(q, k, f, stream=stream, **kw)
    for kw in (dict(q_out=q, k_out=q), dict(q_out=q), dict(q_out=one, k_out=one)):
        with pytest.raises(ValueError, match="in this order"):
            cf.rotary(q, q, f, **kw)
    torch.cuda.synchronize()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    yq, yk = cf.rotary(q, q, f)  # one input for both is fine
    assert torch.equal(yq, yk) and torch.equal(yq, cf.rotary(q, None, f)[0])
    none = torch.empty(0, 2, 64, device="cuda")
    assert cf.rotary(none, none, f, q_out=none, k_out=none)[0] is none
    want = cf.rotary(q, k, f)
    qkv = torch.cat([q, k], dim=1)  # in place in one buffer's rows
    got = cf.rotary(qkv[:, :2], qkv[:, 2:], f, q_out=qkv[:, :2], k_out=qkv[:, 2:])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
