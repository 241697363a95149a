"""Workspace sizes of the attention calls, on the host."""
import pytest

import compensated_fp32_projection_amd as cf


@pytest.mark.parametrize("S,Tk,Hkv,D", [(8192, 8192, 8, 128), (512, 5120, 8, 128), (200, 8000, 12, 64), (1, 100000, 8, 128),
                                        (1000, 1, 4, 64), (1 << 20, 1 << 20, 1, 128)])
def test_prompts_take_what_k_and_v_take(S, Tk, Hkv, D):
    """FP32 K and V of any number of sequences: their FP16 parts, and no
    padding of each sequence (parts of rows apart, at most 34 MB)."""
    kv = 2 * 4 * Tk * Hkv * D
    tile = 64 * Hkv * (8 * D + 8)
    need = cf.cfp32_attention_prompt_workspace_bytes(S, Tk, Hkv, D, cf.KV_F32)
    parts = cf.cfp32_attention_prompt_workspace_bytes(S, Tk, Hkv, D, cf.KV_F16)
    assert kv <= need <= 1.02 * kv + tile + 8 * S * Hkv + parts + 1024 and parts <= 35 << 20
