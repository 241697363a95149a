"""Rows of matrices and tables that step by less than their columns: the helpers never read them as rows one behind the
other (which lie outside the tensor).  On the host, with tensors that have no memory."""
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import compensated_fp32_projection_amd as cf

E = cf.ERR_INVALID_VALUE


def fake(rows, cols, strides, dtype=torch.float32):
    with FakeTensorMode():
        return torch.empty(1000, dtype=dtype, device="cuda").as_strided((rows, cols), strides)


@pytest.fixture(autouse=True)
def quiet():
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")  # addresses of such tensors
        yield


def test_matrices():
    f = (torch.float32,)
    for rows, cols, strides, ld in ((4, 7, (7, 1), 7), (4, 7, (9, 1), 9), (1, 7, (0, 1), 7), (1, 7, (3, 1), 7), (5, 1, (1, 1), 1),
                                    (0, 7, (7, 1), 7), (5, 0, (1, 1), 1), (5, 1, (3, 5), 3)):
        assert cf._mat(fake(rows, cols, strides), f, "x")[1:] == (rows, cols, ld)
    for rows, cols, strides in ((4, 7, (0, 1)), (2, 7, (6, 1)), (2, 2, (1, 1)), (3, 1, (0, 1))):
        with pytest.raises(ValueError, match="overlap"):
            cf._mat(fake(rows, cols, strides), f, "x")


def test_logits():
    """One row for all beams is passed on as it is."""
    f = (torch.float32,)
    assert cf._mat(fake(4, 7, (0, 1)), f, "x", shared=True)[3] == 0
    assert cf._mat(fake(4, 7, (8, 1)), f, "x", shared=True)[3] == 8
    with pytest.raises(ValueError, match="overlap"):
        cf._mat(fake(4, 7, (3, 1)), f, "x", shared=True)


def test_selection_takes_one_row_or_whole_ones():
    if torch.cuda.is_available():
        pytest.skip("would run on made-up pointers")
    a = 1 << 20

    def select(ld):
        return cf.cfp32_beam_select(a, ld, a, None, 3, 4, 1000, 4, 2, a << 1, a << 1, a << 1, None, a, 1 << 40, None)

    assert select(0) == select(1000) == cf.ERR_UNSUPPORTED_DEVICE
    assert select(1) == select(999) == select(-1) == E
