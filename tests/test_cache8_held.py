"""A Cache8 goes on with the memory that it was made of: its attributes are not set anew, and other storages of its
tensors do not reach it."""
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import compensated_fp32_projection_amd as cf


def test_attributes_are_not_set():
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")  # addresses of tensors without memory
        with FakeTensorMode():
            codes, scales = torch.zeros(3, 2, 16, 64, dtype=torch.int8, device="cuda"), torch.zeros(3, 2, 2, device="cuda")
            c = cf.Cache8(codes, codes, scales, scales)
            for name in cf.Cache8.__slots__:
                before = getattr(c, name)
                with pytest.raises(AttributeError, match=name):
                    setattr(c, name, before)
                with pytest.raises(AttributeError, match=name):
                    delattr(c, name)
                assert getattr(c, name) is before
            with pytest.raises(AttributeError):
                c.other = 1


@pytest.mark.gpu
def test_other_storages_do_not_reach_it():
    g = torch.Generator(device="cuda").manual_seed(1)
    pools = [torch.randint(-127, 128, (64, 2, 16, 64), generator=g, device="cuda").to(torch.int8) for _ in range(2)]
    pools += [torch.rand(64, 2, 16, generator=g, device="cuda") for _ in range(2)]
    c = cf.Cache8(*pools)
    q = torch.randn(4, 4, 64, generator=g, device="cuda")
    table = torch.randperm(64, generator=g, device="cuda").to(torch.int32).view(4, 16)
    lens = torch.tensor([256, 100, 7, 255], dtype=torch.int32, device="cuda")
    want = cf.attention8_decode(q, c, table, lens)
    for t in pools + [c.k, c.v_scales]:
        t.data = torch.zeros_like(t)
    # What was given back would come from here.
    filled = [torch.full((64, 2, 16, 64), 1, dtype=torch.int8, device="cuda") for _ in range(8)]
    filled += [torch.full((64, 2, 16), float("nan"), device="cuda") for _ in range(8)]
    assert torch.equal(cf.attention8_decode(q, c, table, lens), want) and len(filled) == 16
