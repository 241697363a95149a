"""Tables of pages whose rows step by less than their width, on the host: what only reads a table takes one row for all
sequences, nothing takes rows that overlap otherwise."""
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import compensated_fp32_projection_amd as cf
import test_attention_abi as paged
import test_cache8_abi as cache8
from test_cache8_abi import lib  # noqa: F401  (a fixture)

E = cf.ERR_INVALID_VALUE


def test_steps():
    def fake(rows, cols, step):
        with FakeTensorMode():
            return torch.empty(1000, dtype=torch.int32, device="cuda").as_strided((rows, cols), (step, 1))

    with warnings.catch_warnings():
        warnings.simplefilter("ignore")
        assert [cf._ld(fake(*a)) for a in ((3, 5, 5), (3, 5, 9), (1, 5, 0), (3, 0, 1), (0, 5, 5))] == [5, 9, 5, 1, 5]
        assert cf._ld(fake(3, 5, 0), shared=True) == 0
        for a in ((3, 5, 0), (3, 5, 4), (2, 1, 0)):
            with pytest.raises(ValueError, match="table: rows overlap"):
                cf._ld(fake(*a))
        for a in ((3, 5, 4), (3, 5, 1)):
            with pytest.raises(ValueError, match="rows overlap"):
                cf._ld(fake(*a), shared=True)


def test_the_calls():
    if torch.cuda.is_available():
        pytest.skip("would run on made-up pointers")
    passed = cf.ERR_UNSUPPORTED_DEVICE
    for name in ("read", "decode"):
        assert cache8.call(name, ld_table=0) == passed
        assert cache8.call(name, ld_table=1) == cache8.call(name, ld_table=-1) == E
    assert paged.call("attention_decode", ld_table=0) == passed
    assert paged.call("attention_decode", ld_table=1) == E
    for name in ("append", "fork", "compact"):
        assert cache8.call(name, ld_table=0) == E
    for name in ("cache_reserve", "cache_append", "cache_fork", "cache_compact"):
        assert paged.call(name, ld_table=0) == E
