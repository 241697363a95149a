"""GPU tests of many packed sequences whose last tiles hold the next ones' first
keys: FP32 K and V through 64-key tiles, against the definition in FP64."""
import numpy as np
import pytest
import torch

from gpu_helpers import note
from test_attention_prompt_gpu import call, dev, make, starts
from test_attention_tiles_gpu import compare

pytestmark = pytest.mark.gpu

LENS = [63, 1, 0, 65, 130, 200, 7, 64] * 6


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (36, 12, 64), (32, 8, 72)])
def test_many_sequences(Hq, Hkv, D, causal):
    note(f"packed sequences {Hq}/{Hkv} x {D} causal={causal}")
    q, k, v = make(D, LENS, LENS, Hq, Hkv, D, "f32")
    cu = starts(LENS)
    compare(call(dev(q), dev(k), dev(v), cu, cu, causal=causal), q, k, v, cu, cu, [Hkv - 1], causal)


@pytest.mark.parametrize("what", ["values", "magnitudes", "nan"])
def test_other_sequences_and_tokens_of_none(what):
    """Every second sequence's keys, and tokens before and behind all
    sequences, changed: the others' results stay (for finite changes, their bits)."""
    note(f"packed neighbours {what}")
    Hq, Hkv, D = 32, 8, 128
    lens = [5] + LENS + [70]
    q, k, v = make(3, lens, lens, Hq, Hkv, D, "f32")
    cu = starts(lens)[1:-1]
    out = torch.zeros(q.shape, device="cuda")
    first = call(dev(q), dev(k), dev(v), cu, cu, out=out)
    change = np.ones(len(k), bool)
    for s in range(0, len(LENS), 2):
        change[cu[s]:cu[s + 1]] = False
    for x in (k, v):
        x[change] = {"values": -x[change], "magnitudes": x[change] * np.float32(1e25), "nan": np.nan}[what]
    out = torch.zeros(q.shape, device="cuda")
    got = call(dev(q), dev(k), dev(v), cu, cu, out=out)
    assert (got[:5] == 0).all() and (got[-70:] == 0).all()
    if what == "nan":
        assert np.isnan(got[5:-70][change[5:-70]]).all()
        assert np.abs(got - first)[~change].max() < 1e-5
    else:
        assert np.array_equal(got[~change], first[~change])
