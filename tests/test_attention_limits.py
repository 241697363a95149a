"""Sizes at the ends of 32 bits, on the host (see test_attention_abi.py): keys
that the kernels' steps beyond the last would not leave within an int32 are
refused."""
import torch

import compensated_fp32_projection_amd as cf
from test_attention_abi import E, call, lib  # noqa: F401

MOST = 2 ** 31 - 2 ** 16


def test_keys_of_a_prompt():
    for n in (MOST + 1, 2 ** 31 - 1):
        assert call("attention_prompt", Tk=n, D=1) == E
        assert cf.cfp32_attention_prompt_workspace_bytes(1, n, 1, 1, cf.KV_F16) == 0
    assert cf.cfp32_attention_prompt_workspace_bytes(1, MOST, 1, 1, cf.KV_F16) > 0
    if not torch.cuda.is_available():  # would run on made-up pointers
        assert call("attention_prompt", Tk=MOST, D=1, kv_type=cf.KV_F16) == cf.ERR_UNSUPPORTED_DEVICE


def test_keys_of_a_cache():
    for W, page in ((MOST // 16 + 1, 16), (2 ** 15, 65536), (2 ** 31 - 1, 1)):
        args = dict(W=W, ld_table=W, page=page, shared_pages=0, k_page=1 << 22, v_page=1 << 22, k_head=1 << 22, v_head=1 << 22)
        assert call("attention_decode", **args) == E, (W, page)
        assert cf.cfp32_attention_decode_workspace_bytes(2, 2, 1, 64, W, page, 0, cf.KV_F16) == 0
    if not torch.cuda.is_available():
        assert call("attention_decode", W=MOST // 16, ld_table=MOST // 16, shared_pages=0) == cf.ERR_UNSUPPORTED_DEVICE
