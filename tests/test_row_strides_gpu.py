"""GPU tests of rows that step by less than their columns: one row for all is read as one, others are refused."""
import numpy as np
import pytest
import torch

import beam_reference as ref
import compensated_fp32_projection_amd as cf
from gpu_helpers import note
from test_beam_gpu import check, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S,beams,V,n", [(1, 4, 1000, 4), (2, 3, 1003, 5), (600, 4, 2050, 3)])
def test_one_row_of_logits_for_all_beams(S, beams, V, n):
    rng = np.random.default_rng(V)
    row = (rng.standard_normal((1, V)) * 3).astype(np.float32)
    scores = (-np.arange(S * beams, dtype=np.float32) * 0.371).reshape(S, beams)
    x = dev(row).expand(S * beams, V)
    note(f"beam one row {S} {beams} {V}")
    want = ref.select(np.repeat(row, S * beams, 0), scores, n)
    check(cf.beam_select(x, dev(scores), n=n), want)
    check(cf.beam_select(x, dev(scores), n=n, workspace=cf.Workspace()), want)  # without the native form
    done = rng.random((S, beams)) < 0.3
    check(cf.beam_select(x, dev(scores), n=n, done=dev(done), eos=1), ref.select(np.repeat(row, S * beams, 0), scores, n, done, 1))


def test_overlapping_rows_are_refused():
    base = torch.zeros(100, device="cuda")
    scores = torch.zeros(1, 3, device="cuda")
    for x in (base.as_strided((3, 10), (9, 1)), base.as_strided((3, 2), (1, 1))):
        for kw in ({}, dict(workspace=cf.Workspace())):
            with pytest.raises(ValueError, match="overlap"):
                cf.beam_select(x, scores, **kw)
    w = torch.zeros(10, 4, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        cf.linear(base[:10].expand(3, 10), w)
    with pytest.raises(ValueError, match="overlap"):
        cf.linear(torch.zeros(3, 10, device="cuda"), w, out=base[:4].expand(3, 4))
