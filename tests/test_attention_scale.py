"""Scales that FP32 does not hold are refused (on the host; see test_attention_abi.py)."""
import pytest
import torch

import compensated_fp32_projection_amd as cf
from test_attention_abi import E, call, lib  # noqa: F401


@pytest.mark.parametrize("name", ["attention_prompt", "attention_decode"])
def test_scales_beyond_fp32(name):
    for scale in (1e39, -1e300, 3.4028236e38, float("inf"), float("nan")):
        assert call(name, scale=scale) == E, scale
    if not torch.cuda.is_available():  # would run on made-up pointers
        for scale in (3.4028234e38, -3.4e38, 1e-60, 0.0):
            assert call(name, scale=scale) == cf.ERR_UNSUPPORTED_DEVICE, scale
