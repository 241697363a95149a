"""Refusals, sizes and empty problems of the attention and cache calls, on the
host (no kernel is launched; see test_abi.py)."""
import os

import pytest
import torch

import compensated_fp32_projection_amd as cf

FAKE, FAKE2 = 1 << 20, 1 << 21  # never dereferenced: these calls fail or return before any device work
E, OK = cf.ERR_INVALID_VALUE, cf.OK


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(cf.LIB_PATH):
        from compensated_fp32_projection_amd import build
        build.build()
    return cf.load_library()


PROMPT = dict(q=FAKE, q_tok=128, q_head=64, k=FAKE, k_tok=64, k_head=64, v=FAKE, v_tok=64, v_head=64, kv_type=0,
              cu_q=FAKE, cu_k=FAKE, out=FAKE, out_tok=128, out_head=64, S=2, Tq=10, Tk=10, Hq=2, Hkv=1, D=64, causal=1,
              scale=0.125, workspace=FAKE, workspace_bytes=1 << 40, stream=None)
DECODE = dict(q=FAKE, q_seq=128, q_head=64, k_pages=FAKE, k_page=1024, k_head=1024, k_tok=64, v_pages=FAKE, v_page=1024,
              v_head=1024, v_tok=64, kv_type=1, P=8, page=16, table=FAKE, ld_table=4, W=4, lens=FAKE, shared_pages=1,
              out=FAKE, out_seq=128, out_head=64, B=2, Hq=2, Hkv=1, D=64, scale=0.125, workspace=FAKE,
              workspace_bytes=1 << 40, stream=None)
POOL = dict(k_pages=FAKE, kp_page=1024, kp_head=1024, kp_tok=64, v_pages=FAKE, vp_page=1024, vp_head=1024, vp_tok=64,
            kv_type=1, P=8, page=16, Hkv=1, D=64)
RESERVE = dict(table=FAKE, ld_table=4, lens=FAKE, cu=FAKE, refs=FAKE, table_out=FAKE2, ld_out=4, refs_out=FAKE2,
               missing=None, S=2, W=4, P=8, page=16, stream=None)
APPEND = dict(k=FAKE, k_tok=64, k_head=64, v=FAKE, v_tok=64, v_head=64, cu=FAKE, lens=FAKE, lens_out=FAKE2, **POOL,
              table=FAKE, ld_table=4, S=2, W=4, T=5, stream=None)
COPY = dict(**POOL, src=FAKE, dst=FAKE2, n=3, stream=None)
FORK = dict(**POOL, table=FAKE, ld_table=4, lens=FAKE, refs=FAKE, parents=FAKE, table_out=FAKE2, ld_out=4,
            lens_out=FAKE2, refs_out=FAKE2, missing=None, S=2, W=4, C=3, workspace=FAKE, workspace_bytes=1 << 20,
            stream=None)
FREE = dict(rows=FAKE, ld_rows=4, refs=FAKE, refs_out=FAKE2, R=2, W=4, P=8, stream=None)
COMPACT = dict(**POOL, table=FAKE, ld_table=4, refs=FAKE, table_out=FAKE2, ld_out=4, refs_out=FAKE2, live=FAKE, S=2,
               W=4, workspace=FAKE, workspace_bytes=1 << 20, stream=None)
CALLS = {"attention_prompt": PROMPT, "attention_decode": DECODE, "cache_reserve": RESERVE, "cache_append": APPEND,
         "cache_copy_pages": COPY, "cache_fork": FORK, "cache_free": FREE, "cache_compact": COMPACT}


def call(name, **changed):
    args = dict(CALLS[name])
    assert set(changed) <= set(args), changed
    args.update(changed)
    return getattr(cf, "cfp32_" + name)(**args)


def test_the_calls_as_they_stand_are_accepted():
    """What every refusal below changes one thing of is refused only for the missing device."""
    if torch.cuda.is_available():
        pytest.skip("would run on made-up pointers")
    for name in CALLS:
        assert call(name) == cf.ERR_UNSUPPORTED_DEVICE, name


REFUSED = {
    "attention_prompt": [
        dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(cu_q=None), dict(cu_k=None), dict(S=-1),
        dict(Tq=-1), dict(Tk=-2), dict(Hq=3, Hkv=2), dict(Hq=2, Hkv=0), dict(D=129), dict(D=-1), dict(kv_type=2),
        dict(Tq=1 << 31), dict(Tk=1 << 31), dict(q=FAKE + 2), dict(k=FAKE + 2), dict(out=FAKE + 1),
        dict(kv_type=1, k=FAKE + 1), dict(q_tok=-1), dict(k_head=-64), dict(out_tok=64), dict(out_head=63),
        dict(out_tok=0), dict(k_tok=1 << 47), dict(scale=float("nan")), dict(scale=float("inf"))],
    "attention_decode": [
        dict(q=None), dict(k_pages=None), dict(v_pages=None), dict(table=None), dict(lens=None), dict(out=None),
        dict(B=-1), dict(Hq=3, Hkv=2), dict(D=129), dict(kv_type=-1), dict(page=0), dict(page=24), dict(page=1 << 17),
        dict(W=-1), dict(ld_table=3), dict(shared_pages=-1), dict(shared_pages=5), dict(P=-1), dict(P=1 << 31),
        dict(W=1 << 28, ld_table=1 << 28), dict(k_page=-1), dict(k_pages=FAKE + 1), dict(kv_type=0, v_pages=FAKE + 2),
        dict(out_seq=64), dict(scale=float("-inf")), dict(v_page=1 << 46)],
    "cache_reserve": [dict(table=None), dict(lens=None), dict(cu=None), dict(refs=None), dict(table_out=None),
                      dict(refs_out=None), dict(S=-1), dict(W=1 << 31), dict(P=-1), dict(page=3), dict(ld_table=3),
                      dict(ld_out=3), dict(table_out=FAKE, ld_out=5)],
    "cache_append": [dict(k=None), dict(v=None), dict(cu=None), dict(lens=None), dict(lens_out=None), dict(lens_out=FAKE),
                     dict(k_pages=None), dict(v_pages=None), dict(table=None), dict(S=-1), dict(T=-1), dict(page=12),
                     dict(kv_type=3), dict(D=200), dict(kp_tok=63), dict(vp_page=1023), dict(kp_page=0), dict(k=FAKE + 1),
                     dict(k_pages=FAKE + 1), dict(ld_table=2)],
    "cache_copy_pages": [dict(src=None), dict(dst=None), dict(k_pages=None), dict(n=-1), dict(page=5), dict(kv_type=9),
                         dict(vp_tok=0), dict(P=-1), dict(D=129)],
    "cache_fork": [dict(table=None), dict(lens=None), dict(refs=None), dict(parents=None), dict(table_out=None),
                   dict(lens_out=None), dict(refs_out=None), dict(k_pages=None), dict(C=-1), dict(workspace=None),
                   dict(workspace_bytes=279), dict(table_out=FAKE), dict(lens_out=FAKE), dict(page=7), dict(ld_out=3),
                   dict(kp_page=100)],
    "cache_free": [dict(rows=None), dict(refs=None), dict(refs_out=None), dict(R=-1), dict(P=-1), dict(ld_rows=3)],
    "cache_compact": [dict(table=None), dict(refs=None), dict(table_out=None), dict(refs_out=None), dict(live=None),
                      dict(workspace=None), dict(workspace_bytes=100), dict(k_pages=None), dict(P=1 << 31),
                      dict(ld_out=3), dict(table_out=FAKE, ld_out=5), dict(page=0), dict(vp_head=8, vp_tok=8)],
}


@pytest.mark.parametrize("name", CALLS)
def test_refusals(name):
    for changed in REFUSED[name]:
        assert call(name, **changed) == E, changed


def test_workspaces_too_small_are_refused():
    for kv in (cf.KV_F32, cf.KV_F16):
        need = cf.cfp32_attention_prompt_workspace_bytes(2, 10, 1, 64, kv)
        if need:
            assert call("attention_prompt", kv_type=kv, workspace_bytes=need - 1) == E
            assert call("attention_prompt", kv_type=kv, workspace=None) == E
        need = cf.cfp32_attention_decode_workspace_bytes(2, 2, 1, 64, 4, 16, 1, kv)
        if need:
            assert call("attention_decode", kv_type=kv, workspace_bytes=need - 1) == E
            assert call("attention_decode", kv_type=kv, workspace=None) == E


def test_workspace_queries_of_refused_sizes():
    assert cf.cfp32_attention_prompt_workspace_bytes(-1, 10, 1, 64, 0) == 0
    assert cf.cfp32_attention_prompt_workspace_bytes(1, 10, 1, 129, 0) == 0
    assert cf.cfp32_attention_prompt_workspace_bytes(1, 10, 1, 64, 5) == 0
    assert cf.cfp32_attention_prompt_workspace_bytes(2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 128, 0) == 0
    assert cf.cfp32_attention_decode_workspace_bytes(1, 3, 2, 64, 4, 16, 0, 0) == 0
    assert cf.cfp32_attention_decode_workspace_bytes(1, 2, 2, 64, 4, 17, 0, 0) == 0
    assert cf.cfp32_attention_decode_workspace_bytes(1, 2, 2, 64, 4, 16, 5, 0) == 0
    assert cf.cfp32_attention_decode_workspace_bytes(2 ** 31 - 1, 2 ** 30, 1, 64, 4, 16, 0, 0) == 0
    assert cf.cfp32_cache_fork_workspace_bytes(-1) == 0 and cf.cfp32_cache_compact_workspace_bytes(-1) == 0


def test_empty_problems_are_no_ops():
    assert call("attention_prompt", S=0, q=None, out=None, cu_q=None, cu_k=None) == OK
    assert call("attention_prompt", Tq=0, q=None) == OK
    assert call("attention_prompt", Hq=0, Hkv=0) == OK
    assert call("attention_prompt", D=0) == OK
    assert call("attention_decode", B=0, q=None, table=None, lens=None) == OK
    assert call("attention_decode", D=0) == OK
    assert call("cache_reserve", S=0, P=0, refs=None, refs_out=None) == OK
    assert call("cache_append", S=0, cu=None) == OK
    assert call("cache_copy_pages", n=0, src=None, dst=None) == OK
    assert call("cache_copy_pages", P=0, k_pages=None, v_pages=None) == OK
    assert call("cache_fork", C=0, P=0, refs=None, refs_out=None) == OK
    assert call("cache_free", P=0, refs=None, refs_out=None) == OK


def test_helpers_check_their_tensors():
    """The tensor helpers refuse what is not on a GPU, of another type, or of another shape, before any call."""
    x = torch.zeros(4, 2, 64)
    i = torch.zeros(3, dtype=torch.int32)
    pages = torch.zeros(3, 2, 16, 64)
    with pytest.raises(TypeError):
        cf.attention_prompt(x, x, x, i)
    with pytest.raises(TypeError):
        cf.attention_decode(x, pages, pages, torch.zeros(4, 2, dtype=torch.int32), i)
    with pytest.raises(TypeError):
        cf.cache_append(x, x, i, pages, pages, i, i)
    with pytest.raises(TypeError):
        cf.cache_copy_pages(pages, pages, i, i)
    with pytest.raises(TypeError):
        cf.cache_reserve(i[None].long(), i, i, i, 16)
