"""Refusals and empty problems of the beam search calls, on the host (no kernel is launched)."""
import pytest
import torch

import compensated_fp32_projection_amd as cf

FAKE, FAKE2 = 1 << 20, 1 << 21  # never dereferenced
E, OK = cf.ERR_INVALID_VALUE, cf.OK

SELECT = dict(logits=FAKE, ld=1000, scores=FAKE, done=FAKE, S=3, beams=4, V=1000, n=4, eos=2, parents=FAKE2, tokens=FAKE2,
              scores_out=FAKE2, done_out=FAKE2, workspace=FAKE, workspace_bytes=1 << 40, stream=None)
REORDER = dict(states=FAKE, stride=100, out=FAKE2, out_stride=100, parents=FAKE, rows=5, n=7, row_bytes=100, stream=None)


def select(**changed):
    assert set(changed) <= set(SELECT)
    return cf.cfp32_beam_select(**{**SELECT, **changed})


def reorder(**changed):
    assert set(changed) <= set(REORDER)
    return cf.cfp32_beam_reorder(**{**REORDER, **changed})


def test_the_calls_as_they_stand_are_accepted():
    if torch.cuda.is_available():
        pytest.skip("would run on made-up pointers")
    assert select() == cf.ERR_UNSUPPORTED_DEVICE
    assert select(done=None, done_out=None, eos=-1, n=64, beams=64) == cf.ERR_UNSUPPORTED_DEVICE
    assert reorder() == cf.ERR_UNSUPPORTED_DEVICE
    assert reorder(stride=0) == cf.ERR_UNSUPPORTED_DEVICE
    assert reorder(rows=0, states=None) == cf.ERR_UNSUPPORTED_DEVICE


@pytest.mark.parametrize("changed", [
    dict(logits=None), dict(scores=None), dict(parents=None), dict(tokens=None), dict(scores_out=None), dict(workspace=None),
    dict(S=-1), dict(beams=0), dict(beams=65), dict(n=0), dict(n=65), dict(V=0), dict(V=1 << 31), dict(ld=999), dict(ld=1 << 46),
    dict(scores_out=FAKE), dict(done_out=FAKE), dict(scores_out=FAKE, done=None),
    dict(logits=FAKE + 2), dict(workspace_bytes=100), dict(S=1 << 30), dict(eos=1 << 40), dict(eos=-(1 << 40))])
def test_refused_selections(changed):
    assert select(**changed) == E


@pytest.mark.parametrize("changed", [
    dict(states=None), dict(out=None), dict(parents=None), dict(rows=-1), dict(n=-1), dict(row_bytes=-1), dict(out_stride=99),
    dict(stride=-1), dict(out=FAKE), dict(n=1 << 31), dict(stride=1 << 47), dict(row_bytes=1 << 47, out_stride=1 << 47)])
def test_refused_reorders(changed):
    assert reorder(**changed) == E


def test_workspace_queries_and_empty_problems():
    assert cf.cfp32_beam_select_workspace_bytes(3, 4, 1000, 4) > 0
    for bad in ((-1, 4, 1000, 4), (0, 4, 1000, 4), (3, 0, 1000, 4), (3, 65, 1000, 4), (3, 4, 0, 4), (3, 4, 1000, 0),
                (3, 4, 1000, 65), (3, 4, 1 << 31, 4), (1 << 31, 4, 10, 4)):
        assert cf.cfp32_beam_select_workspace_bytes(*bad) == 0
    need = cf.cfp32_beam_select_workspace_bytes(3, 4, 1000, 4)
    assert select(workspace_bytes=need - 1) == E
    assert select(S=0, logits=None, scores=None, workspace=None) == OK
    assert reorder(n=0, states=None, out=None, parents=None) == OK
    assert reorder(row_bytes=0) == OK


def test_the_helpers_check_their_tensors():
    x, i = torch.zeros(4, 10), torch.zeros(4, dtype=torch.int32)
    for f in (lambda: cf.beam_select(x, x[:2, :2]), lambda: cf.beam_reorder(x, i)):
        with pytest.raises(TypeError):
            f()
