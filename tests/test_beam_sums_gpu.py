"""GPU tests of the sums behind a beam's log-probabilities, at logits that put all roundings on one side.

With u = 2^-24: a logit's term is 2^f 2^n, |f| <= 1/2.  f has two roundings of half its last place (2 u / 8 below 1/4,
2 u / 4 from there on), times ln 2; 2^f is off by one unit in its last place, 2 u / 2^f from f = 0 on and u / 2^f below:
together 2.03 u at most, at f = 1/4 (2 / 1.189 + 0.347), and less than 2.01 u below it.  Two terms are added in FP32, u;
pairs in FP64; each 512 or 2048 logits' sum is rounded to FP32, u.  All of them on one side put a sum, and so its
logarithm, off by 4.03 u.  A score is that and one rounding to FP32 off.
"""
import numpy as np
import pytest
import torch

import compensated_fp32_projection_amd as cf
from gpu_helpers import note

pytestmark = pytest.mark.gpu

BOUND = 4.03 * 2.0 ** -24


def compare(logits, n=1):
    """One sequence to a row."""
    x = logits.astype(np.float64)
    most = x.max(axis=1, keepdims=True)
    logp = x - (most + np.log(np.exp(x - most).sum(axis=1, keepdims=True)))
    want = -np.sort(-logp, axis=1)[:, :n]
    got = cf.beam_select(torch.from_numpy(logits).cuda(), torch.zeros(len(logits), 1, device="cuda"), n=n)[2].cpu().numpy()
    off = np.abs(got - want) - 2.0 ** -24 * np.abs(want)
    assert off.max() <= BOUND, off.max() / BOUND


@pytest.mark.parametrize("V,rows", [(2048, 2100), (2047, 2100), (512, 3), (513, 3), (20000, 250), (50001, 2)])
@pytest.mark.parametrize("high", [0.0, 12.3, -7.1])
def test_a_peak_over_a_constant(high, V, rows):
    """One logit, and all others equal, 0.1 to 20 below it."""
    rng = np.random.default_rng(V)
    logits = np.zeros((rows, V), np.float32)
    logits[:] = (np.float32(high) - rng.uniform(0.1, 20, (rows, 1))).astype(np.float32)
    logits[0], logits[1] = np.float32(high - 13.8), np.float32(high - 8.7)
    logits[np.arange(rows), rng.integers(0, V, rows)] = high
    note(f"beam sums {V} {rows} {high}")
    compare(logits)


@pytest.mark.parametrize("shift", [0.0, 1e3, -3e4, 2.0 ** 19 - 8, 2.0 ** 19 + 8, -2.0 ** 22, 1e7, 1e12, 3e38])
def test_steps_of_few_values(shift):
    """A handful of values, many times each, near zero and far from it."""
    rng = np.random.default_rng(2)
    values = np.float32(rng.uniform(-15, 0, 5))
    logits = (values[rng.integers(0, 5, (40, 3001))] + np.float32(shift)).astype(np.float32)
    note(f"beam sums shift {shift}")
    compare(logits, n=3)


def test_extremes_beside_ordinary_ones():
    rng = np.random.default_rng(3)
    logits = rng.standard_normal((6, 2500)).astype(np.float32)
    low = np.finfo(np.float32).min
    logits[0, ::2] = -np.inf
    logits[1, ::2] = low
    logits[2] += np.float32(2.0 ** 18)
    logits[3, 7] = np.finfo(np.float32).max
    logits[4, 9] = np.finfo(np.float32).max
    logits[4, 10:] = low
    logits[5] = np.float32(1e-40)
    note("beam sums extremes")
    compare(logits, n=1)
