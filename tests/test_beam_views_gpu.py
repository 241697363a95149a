"""GPU tests of beam_reorder with views whose values are not those in memory: refused, not moved as they lie there."""
import pytest
import torch

import compensated_fp32_projection_amd as cf
from gpu_helpers import note

pytestmark = pytest.mark.gpu


def test_conjugate_and_negated_views():
    x = torch.randn(5, 6, dtype=torch.complex64, device="cuda")
    parents = torch.tensor([4, 0, -1, 2], dtype=torch.int32, device="cuda")
    one = torch.randn(5, 1, dtype=torch.complex64, device="cuda").conj().imag  # negated when read
    assert x.conj().is_conj() and one.is_neg()
    note("beam reorder views")
    for states in (x.conj(), one):
        for kw in ({}, dict(out=torch.empty(4, *states.shape[1:], dtype=states.dtype, device="cuda"))):
            with pytest.raises(ValueError, match="states: a view"):
                cf.beam_reorder(states, parents, **kw)
    with pytest.raises(ValueError, match="out: a view"):
        cf.beam_reorder(x, parents, out=torch.empty(4, 6, dtype=torch.complex64, device="cuda").conj())
    for states in (x, x.conj().resolve_conj(), one.resolve_neg()):
        want = states[parents.clamp(min=0).long()]
        want[2] = 0
        assert torch.equal(cf.beam_reorder(states, parents), want)
