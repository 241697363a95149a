"""GPU tests of long prompts (64-key tiles) whose K and V differ in magnitude
from token to token: a row's result is FP32-grade whatever the keys it does not
see, or gives no weight, hold (definition in FP64, tolerance derived in
attention_reference.py)."""
import numpy as np
import pytest

from gpu_helpers import note
from test_attention_prompt_gpu import call, dev, make, starts
from test_attention_tiles_gpu import compare

pytestmark = pytest.mark.gpu

SHAPES = {
    # sequences, Hq, Hkv, D, head compared
    "four_waves": ([1100], 12, 12, 64, 7),
    "parts": ([1500], 12, 12, 64, 3),                                          # keys in parts, joined
    "eight_waves": ([290, 310, 270, 300, 305, 295, 340, 290], 32, 8, 128, 5),
    "seventy_tiles": ([4500], 4, 4, 64, 2),
    "odd_dim": ([900, 700], 16, 8, 80, 6),
}

FORMS = ["four_waves", "parts", "eight_waves", "odd_dim"]


def run(shape, seed, change, causal=True):
    """A prompt of that shape whose q, k, v of every sequence went through `change`, against the definition."""
    lens, Hq, Hkv, D, head = SHAPES[shape]
    q, k, v = make(seed, lens, lens, Hq, Hkv, D, "f32")
    cu = starts(lens)
    for a, b in zip(cu[:-1], cu[1:]):
        change(q[a:b], k[a:b], v[a:b])
    compare(call(dev(q), dev(k), dev(v), cu, cu, causal=causal), q, k, v, cu, cu, [head], causal=causal)


@pytest.mark.parametrize("shape", FORMS)
def test_tiles_of_rising_values(shape):
    """Rows that see the first tile only, before tiles of 2^200 times its values."""
    note(f"rising values {shape}")

    def change(q, k, v):
        v[:64] *= np.float32(1e-30)
        v[64:] *= np.float32(1e30)

    run(shape, 51, change)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", FORMS)
def test_tiles_of_large_values_without_weight(shape, causal):
    """Large values whose keys weigh nothing, before small ones."""
    note(f"large weightless tiles {shape} causal={causal}")

    def change(q, k, v):
        np.abs(q, out=q)
        k[:64] = -40
        v[:64] *= np.float32(1e30)
        v[64:] *= np.float32(1e-30)

    run(shape, 52, change, causal)


def test_values_fall_and_rise_between_tiles():
    """Magnitudes over all of FP32's range from tile to tile."""
    note("values fall and rise")
    f = np.float32(10.0) ** np.random.default_rng(53).integers(-34, 35, 17).astype(np.float32)

    def change(q, k, v):
        v *= np.resize(f.repeat(64), len(v))[:, None, None]

    run("four_waves", 53, change)


@pytest.mark.parametrize("what", ["key", "value"])
def test_one_large_token_far_on(what):
    """In the seventieth tile."""
    note(f"one large {what} far on")

    def change(q, k, v):
        (k if what == "key" else v)[4450] *= np.float32(1e12)

    run("seventy_tiles", 59, change)


@pytest.mark.parametrize("factor", [1e6, 1e8, 1e12, 1e30])
@pytest.mark.parametrize("what", ["key", "value"])
@pytest.mark.parametrize("shape", FORMS)
def test_one_large_token(shape, what, factor):
    """One token's keys or values multiplied: the rows before it do not see it."""
    note(f"one large {what} x {factor} {shape}")

    def change(q, k, v):
        (k if what == "key" else v)[180] *= np.float32(factor)

    run(shape, 54, change)


@pytest.mark.parametrize("what", ["key", "value"])
@pytest.mark.parametrize("shape", FORMS)
def test_one_small_token(shape, what):
    """One token's keys or values next to nothing; one row sees it alone."""
    note(f"one small {what} {shape}")

    def change(q, k, v):
        (k if what == "key" else v)[0] *= np.float32(1e-20)

    run(shape, 55, change)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("shape", FORMS)
def test_large_tokens_without_weight(shape, causal):
    """Every second token has large values, and keys (some of them large) that give it no weight."""
    note(f"large weightless tokens {shape} causal={causal}")

    def change(q, k, v):
        np.abs(q, out=q)
        k[1::4] = -40
        k[3::4] = -1e15
        v[1::2] *= np.float32(1e20)

    run(shape, 56, change, causal)


def test_tokens_of_every_magnitude():
    """Values over all of FP32's range from token to token, and keys of different magnitudes."""
    note("tokens of every magnitude")
    rng = np.random.default_rng(57)

    def change(q, k, v):
        n = len(v)
        v *= np.float32(10.0) ** rng.integers(-34, 35, n).astype(np.float32)[:, None, None]
        k *= np.float32(10.0) ** rng.integers(-9, 1, n).astype(np.float32)[:, None, None]
        v[rng.integers(0, n, n // 9)] = 0
        k[rng.integers(0, n, n // 9)] = 0

    run("four_waves", 57, change)
    run("eight_waves", 58, change)
