"""The layer of examples/attention_layer.py: projection, rotary packing,
attention and the paged cache together, against the layer in FP64."""
import os
import sys

import pytest
import torch

from gpu_helpers import note

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


# Errors of the FP32-grade steps relative to the largest output, each at most a
# few steps of FP32 on sums of up to 768 terms: 768 * 2^-24 = 4.6e-5.
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("tokens,samples", [(200, 6), (64, 1), (37, 3), (16, 4)])
def test_layer(tokens, samples, dtype):
    import attention_layer
    note(f"attention layer {tokens} {samples} {dtype}")
    assert attention_layer.run(tokens=tokens, samples=samples, dtype=dtype) <= 4.6e-5
