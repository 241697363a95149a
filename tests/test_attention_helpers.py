"""The tensor helpers' refusals, on the CPU: whatever is not a plain call falls
through the native form to the checks that say what is wrong."""
import pytest
import torch

import compensated_fp32_projection_amd as cf


def ints(*x):
    return torch.tensor(x, dtype=torch.int32)


def test_cpu_tensors_are_refused():
    q, cu = torch.zeros(4, 2, 64), ints(0, 4)
    pool = torch.zeros(4, 2, 16, 64)
    table, lens, refs = torch.zeros(1, 4, dtype=torch.int32), ints(3), torch.zeros(4, dtype=torch.int32)
    for f in (lambda: cf.attention_prompt(q, q, q, cu), lambda: cf.attention_decode(q, pool, pool, table, lens),
              lambda: cf.cache_append(q, q, cu, pool, pool, table, lens),
              lambda: cf.cache_fork(pool, pool, table, lens, refs, ints(0)),
              lambda: cf.cache_compact(pool, pool, table, refs), lambda: cf.cache_copy_pages(pool, pool, ints(0), ints(1))):
        with pytest.raises(TypeError):
            f()


def test_native_form_declines_what_is_not_plain():
    n = cf._native()
    q, cu = torch.zeros(4, 2, 64), ints(0, 4)
    assert n.attention_prompt(q, q, q, cu, None, True, None, None) is None       # not GPU tensors
    assert n.attention_prompt(q, q, q, cu) is None                              # not its arguments
    assert n.attention_prompt(1, 2, 3, 4, None, True, None, None) is None
    assert n.attention_decode(q, None, q, cu, cu, 0, None, None) is None
    assert n.attention_decode(q, q, q, cu, cu, 1 << 70, None, None) is None
    assert n.cache_reserve(cu, cu, cu, cu, 1 << 70) is None
    assert n.cache_reserve(None, cu, cu, cu, 16) is None
    assert n.cache_append(*[None] * 7) is None and n.cache_fork(*[None] * 6) is None
    assert n.cache_free(None, cu) is None and n.cache_free(cu, None) is None and n.cache_compact(q, q, cu, cu) is None


def test_native_form_binds_only_whole_tables():
    with pytest.raises(TypeError):
        cf._native().bind((1, 2), None, None)
