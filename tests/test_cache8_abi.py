"""Refusals and empty problems of the 8-bit cache's calls, on the host (no kernel is launched)."""
import ctypes
import os

import pytest
import torch

import compensated_fp32_projection_amd as cf

FAKE, FAKE2 = 1 << 20, 1 << 21  # never dereferenced
E, OK = cf.ERR_INVALID_VALUE, cf.OK


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(cf.LIB_PATH):
        from compensated_fp32_projection_amd import build
        build.build()
    return cf.load_library()


CACHE = dict(k=FAKE, v=FAKE, k_page=2048, k_head=1024, k_tok=64, v_page=2048, v_head=1024, v_tok=64, k_scales=FAKE,
             v_scales=FAKE, ks_page=4, ks_head=2, vs_page=4, vs_head=2, P=8, Hkv=2, page=16, block=8, D=64, code_type=0)
APPEND = dict(k=FAKE, k_tok=128, k_head=64, v=FAKE, v_tok=128, v_head=64, cu=FAKE, lens=FAKE, lens_out=FAKE2, cache=None,
              table=FAKE, ld_table=4, S=2, W=4, T=5, stream=None)
READ = dict(cache=None, table=FAKE, ld_table=4, first=None, cu=FAKE, k=FAKE, k_tok=128, k_head=64, v=FAKE, v_tok=128,
            v_head=64, out_type=0, S=2, W=4, T=5, stream=None)
COPY = dict(cache=None, src=FAKE, dst=FAKE2, n=3, stream=None)
FORK = dict(cache=None, table=FAKE, ld_table=4, lens=FAKE, refs=FAKE, parents=FAKE, table_out=FAKE2, ld_out=4,
            lens_out=FAKE2, refs_out=FAKE2, missing=None, S=2, W=4, C=3, workspace=FAKE, workspace_bytes=1 << 20,
            stream=None)
COMPACT = dict(cache=None, table=FAKE, ld_table=4, refs=FAKE, table_out=FAKE2, ld_out=4, refs_out=FAKE2, live=FAKE, S=2,
               W=4, workspace=FAKE, workspace_bytes=1 << 20, stream=None)
DECODE = dict(q=FAKE, q_seq=256, q_head=64, cache=None, table=FAKE, ld_table=400, W=400, lens=FAKE, out=FAKE2, out_seq=256,
              out_head=64, B=2, Hq=4, scale=0.125, workspace=FAKE, workspace_bytes=1 << 40, stream=None)
CALLS = {"append": APPEND, "read": READ, "copy_pages": COPY, "fork": FORK, "compact": COMPACT,
         "decode": DECODE}


def call(name, cache=None, no_cache=False, **changed):
    """The call with some arguments changed, and (cache=) some fields of the pools' description."""
    args = dict(CALLS[name])
    assert set(changed) <= set(args) and set(cache or {}) <= set(CACHE)
    args.update(changed)
    desc = cf.Cache8Desc(**{**CACHE, **(cache or {})})
    args["cache"] = None if no_cache else ctypes.addressof(desc)
    return getattr(cf, "cfp32_attention8_decode" if name == "decode" else "cfp32_cache8_" + name)(**args)


@pytest.mark.parametrize("name", CALLS)
def test_the_calls_as_they_stand_are_accepted(name):
    if torch.cuda.is_available():
        pytest.skip("would run on made-up pointers")
    assert call(name) == cf.ERR_UNSUPPORTED_DEVICE
    assert call(name, cache=dict(code_type=1, block=16, ks_head=1, vs_head=1)) == cf.ERR_UNSUPPORTED_DEVICE
    assert call(name, cache=dict(P=0, k=None, v=None, k_scales=None, v_scales=None)) in (cf.ERR_UNSUPPORTED_DEVICE, OK)


# What each call refuses in the description: pools that are only read may overlap themselves.
BOTH = [dict(k=None), dict(v=None), dict(k_scales=None), dict(v_scales=None), dict(k_scales=FAKE + 2), dict(P=-1),
        dict(P=1 << 31), dict(Hkv=-1), dict(Hkv=65536), dict(page=0), dict(page=24), dict(page=1 << 17), dict(block=0),
        dict(block=3), dict(block=32), dict(block=-8), dict(D=129), dict(D=-1), dict(code_type=2), dict(code_type=-1),
        dict(k_page=-1), dict(v_head=-1), dict(k_tok=-64), dict(ks_page=-1), dict(vs_head=-2), dict(v_page=1 << 46)]
WRITTEN = [dict(k_tok=63), dict(v_page=2047), dict(k_head=0), dict(ks_head=1), dict(vs_page=3), dict(ks_page=0)]


@pytest.mark.parametrize("name", CALLS)
def test_refused_pools(name):
    assert call(name, no_cache=True) == E
    for bad in BOTH + (WRITTEN if name not in ("read", "decode") else []):
        assert call(name, cache=bad) == E, bad


REFUSED = {
    "append": [dict(k=None), dict(v=None), dict(cu=None), dict(lens=None), dict(lens_out=None), dict(lens_out=FAKE),
               dict(table=None), dict(ld_table=3), dict(S=-1), dict(T=-1), dict(W=-1), dict(W=1 << 28, ld_table=1 << 28),
               dict(k=FAKE + 2), dict(k_tok=-1), dict(v_tok=1 << 47)],
    "read": [dict(table=None), dict(cu=None), dict(k=None), dict(v=None), dict(out_type=2), dict(out_type=-1), dict(S=-1),
             dict(T=1 << 31), dict(W=1 << 28, ld_table=1 << 28), dict(ld_table=3), dict(k=FAKE + 2),
             dict(out_type=1, v=FAKE + 1), dict(k_tok=127), dict(v_head=63), dict(k_tok=0), dict(v_tok=-1)],
    "copy_pages": [dict(src=None), dict(dst=None), dict(n=-1), dict(n=1 << 31)],
    "fork": [dict(table=None), dict(lens=None), dict(refs=None), dict(parents=None), dict(table_out=None),
             dict(lens_out=None), dict(refs_out=None), dict(C=-1), dict(workspace=None), dict(workspace_bytes=279),
             dict(table_out=FAKE), dict(lens_out=FAKE), dict(ld_out=3), dict(S=-1), dict(W=1 << 28, ld_table=1 << 28)],
    "compact": [dict(table=None), dict(refs=None), dict(table_out=None), dict(refs_out=None), dict(live=None),
                dict(workspace=None), dict(workspace_bytes=100), dict(ld_out=3), dict(table_out=FAKE, ld_out=5),
                dict(S=-1)],
    "decode": [dict(q=None), dict(table=None), dict(lens=None), dict(out=None), dict(B=-1), dict(Hq=3), dict(Hq=-4),
               dict(W=-1), dict(ld_table=399), dict(W=1 << 28, ld_table=1 << 28), dict(q=FAKE + 2), dict(out=FAKE + 1),
               dict(q_seq=-1), dict(out_seq=255), dict(out_head=63), dict(scale=float("nan")), dict(scale=1e39),
               dict(workspace=None), dict(workspace_bytes=100), dict(B=1 << 30, Hq=1 << 30)],
}


@pytest.mark.parametrize("name", CALLS)
def test_refusals(name):
    for changed in REFUSED[name]:
        assert call(name, **changed) == E, changed


def test_empty_problems_are_no_ops():
    assert call("append", S=0, cu=None, table=None) == OK
    assert call("read", T=0, k=None, v=None) == OK
    assert call("read", S=0, cu=None) == OK
    assert call("copy_pages", n=0, src=None, dst=None) == OK
    assert call("copy_pages", cache=dict(P=0)) == OK
    assert call("fork", cache=dict(P=0), C=0, refs=None, refs_out=None) == OK
    assert call("decode", B=0, q=None, table=None, lens=None) == OK
    assert call("decode", cache=dict(D=0), workspace=None) == OK
    assert call("decode", cache=dict(Hkv=0), Hq=0) == OK


def test_workspace_queries():
    need = cf.cfp32_attention8_decode_workspace_bytes
    assert need(2, 4, 2, 64, 4, 16) == 0  # one step of keys: no parts
    assert need(1, 32, 8, 128, 1024, 64) > 0
    for bad in ((-1, 4, 2, 64, 4, 16), (2, 3, 2, 64, 4, 16), (2, 4, 2, 129, 4, 16), (2, 4, 2, 64, -1, 16), (2, 4, 2, 64, 4, 17),
                (2, 4, 2, 64, 1 << 28, 16), (2 ** 31 - 1, 2 ** 30, 1, 64, 4, 16), (2, 65536, 65536, 64, 4, 16)):
        assert need(*bad) == 0, bad


def test_the_description_is_the_headers():
    """The fields of the C struct, in order, all of eight bytes."""
    here = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(here, "include", "cfp32.h")).read()
    body = text[text.index("typedef struct {\n    void *k, *v;"):text.index("} cfp32_cache8;")]
    names = []
    for line in body.split("\n")[1:]:
        decl = line.split("/*")[0].strip().rstrip(";")
        for word in decl.split(",") if decl else []:
            names.append(word.replace("*", " ").split()[-1])
    assert names == [f[0] for f in cf.Cache8Desc._fields_]
    assert ctypes.sizeof(cf.Cache8Desc) == 8 * len(names)


def test_the_helpers_check_their_tensors():
    codes, scales = torch.zeros(3, 2, 16, 64, dtype=torch.int8), torch.zeros(3, 2, 2)
    with pytest.raises(TypeError):
        cf.Cache8(codes, codes, scales, scales)  # not on a GPU
    i = torch.zeros(3, dtype=torch.int32)
    for f in (lambda: cf.cache8_append(codes, codes, i, codes, i, i), lambda: cf.cache8_read(codes, i, i, 3),
              lambda: cf.cache8_fork(codes, i, i, i, i), lambda: cf.cache8_compact(codes, i, i),
              lambda: cf.cache8_copy_pages(codes, i, i), lambda: cf.attention8_decode(scales, codes, i, i)):
        with pytest.raises(TypeError):
            f()
