"""The example of examples/beam_search.py: projection, rotary positions, the 8-bit
cache written, read, forked and attended to, selection and reordering, together."""
import os
import sys

import numpy as np
import pytest
import torch

import beam_reference as ref
import compensated_fp32_projection_amd as cf
from gpu_helpers import note

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


# Attention against FP64 on the values that the cache stands for, read back rounded to FP32: sums of up to 120 terms of
# 64 products, a few steps of FP32 each: 2^-24 * 768 = 4.6e-5 of the largest value, as for the other cache's example.
@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("prompts,beams,block", [((70, 33, 101), 4, 8), ((16,), 1, 16), ((31, 64), 7, 1)])
def test_search(prompts, beams, block, dtype):
    import beam_search
    note(f"beam search {prompts} {beams} {block} {dtype}")
    history, scores, off = beam_search.run(prompts=prompts, beams=beams, block=block, dtype=dtype)
    assert off <= 4.6e-5
    assert history.shape == (len(prompts), beams, 12) and bool((scores[:, :-1] >= scores[:, 1:]).all())


def test_selections_are_the_definitions(monkeypatch):
    """Every selection of a search against FP64 on its own logits, and pages counted as the running tables name them."""
    import beam_search
    note("beam search selections")
    seen = []
    select = cf.beam_select

    def checked(logits, scores, n=None, done=None, eos=-1):
        got = select(logits, scores, n=n, done=done, eos=eos)
        want = ref.select(logits.cpu().numpy(), scores.cpu().numpy(), n, None if done is None else done.cpu().numpy(), eos)
        if want[4] > 2e-6:  # nearer totals of different beams may change places
            assert np.array_equal(got[0].cpu().numpy(), want[0]) and np.array_equal(got[1].cpu().numpy(), want[1])
            seen.append(1)
        return got

    reorder = beam_search.Cache.reorder

    def counted(self, parents):
        reorder(self, parents)
        table = self.table.cpu().numpy()
        want = np.bincount(table[table >= 0], minlength=len(self.refs))
        assert np.array_equal(self.refs.cpu().numpy(), want)

    monkeypatch.setattr(cf, "beam_select", checked)
    monkeypatch.setattr(beam_search.Cache, "reorder", counted)
    beam_search.run(prompts=(40, 9), beams=5, steps=20, vocab=300)
    assert len(seen) >= 10
