"""GPU tests that attention is FP32-grade on every path: its RMS error against
FP64 beside that of plain FP32 (attention_precision.py)."""
import numpy as np
import pytest

import attention_precision as ap
from gpu_helpers import note
from test_attention_decode_gpu import call as decode_call
from test_attention_decode_gpu import make as decode_make
from test_attention_prompt_gpu import call, dev, make, starts

import attention_reference as ref

pytestmark = pytest.mark.gpu

PROMPTS = [
    # rows, keys, Hq, Hkv, D, kv
    ([37], [37], 12, 12, 64, "f32"), ([37], [37], 4, 2, 128, "f16"),                   # 16-row blocks
    ([512], [512], 12, 12, 64, "f32"), ([300], [300], 12, 12, 64, "f16"),
    ([16], [716], 8, 2, 128, "f32"), ([16], [716], 8, 2, 128, "f16"),                  # keys in parts
    ([1100], [1100], 12, 12, 64, "f32"), ([500], [500], 32, 8, 128, "f32"),            # tiles
    ([900, 700], [900, 700], 16, 8, 80, "f32"), ([1500], [1500], 12, 12, 64, "f32"),
    ([100, 120, 90, 110], [100, 120, 90, 110], 32, 8, 128, "f16"), ([1600], [1600], 12, 12, 64, "f16"),
    ([290, 310, 270, 300, 305, 295, 340, 290], [290, 374, 270, 300, 305, 295, 340, 290], 32, 8, 128, "f32"),  # eight waves
    ([1200, 1150], [1200, 1281], 64, 16, 64, "f32"), ([1200, 1150], [1200, 1281], 64, 16, 128, "f16"),
]


def grade(mine, plain, what):
    note(f"{what}: RMS {mine:.2e}, plain FP32 {plain:.2e}, {mine / plain:.2f} times")
    assert mine <= ap.RATIO * plain, f"{what}: RMS error {mine:.3g}, plain FP32's {plain:.3g}"


@pytest.mark.parametrize("case,varied", [(c, x) for c in PROMPTS for x in (False, True) if not x or c[5] == "f32"],
                         ids=lambda c: f"{len(c[0])}x{max(c[0])}h{c[2]}-{c[3]}d{c[4]}{c[5]}" if isinstance(c, tuple) else "")
def test_prompts(case, varied):
    """On keys and values of one magnitude, and of magnitudes that differ from token to token (FP32)."""
    lq, lk, Hq, Hkv, D, kv = case
    note(f"precision of prompt {lq} {lk} {Hq}/{Hkv} x {D} {kv} varied={varied}")
    q, k, v = make(sum(lk) + D, lq, lk, Hq, Hkv, D, kv)
    if varied:
        rng = np.random.default_rng(9)
        k *= np.float32(2.0) ** rng.integers(-20, 1, len(k)).astype(np.float32)[:, None, None]
        v *= np.float32(2.0) ** rng.integers(-3, 20, len(v)).astype(np.float32)[:, None, None]
    cu_q, cu_k = starts(lq), starts(lk)
    got = call(dev(q), dev(k), dev(v), cu_q, cu_k)
    for s in sorted({0, len(lq) - 1}):
        a, b, a2, b2 = cu_q[s], cu_q[s + 1], cu_k[s], cu_k[s + 1]
        limits = np.arange(b - a) + (b2 - a2) - (b - a) + 1
        h = Hq - 1
        grade(*ap.errors(got[a:b, h], q[a:b, h], k[a2:b2, -1], v[a2:b2, -1], limits, D ** -0.5), f"sequence {s}")


DECODES = [
    # lens, shared pages, page, Hq, Hkv, D, kv
    ([130] * 4, 0, 16, 32, 8, 128, "f16"), ([300, 256, 200, 280], 0, 64, 12, 12, 64, "f32"),
    ([4000, 3900], 0, 16, 16, 2, 128, "f16"), ([2000] * 8, 0, 16, 4, 4, 64, "f32"),
    ([2333] * 12, 125, 16, 12, 12, 64, "f32"), ([400] * 12, 6, 64, 8, 2, 128, "f16"),
    ([5952 + 3 * i for i in range(20)], 93, 64, 64, 8, 128, "f16"), ([12100] * 30, 378, 32, 14, 2, 64, "f16"),  # tiles
]


@pytest.mark.parametrize("case", DECODES, ids=lambda c: f"{len(c[0])}x{max(c[0])}s{c[1]}p{c[2]}h{c[3]}-{c[4]}d{c[5]}{c[6]}")
def test_decodes(case):
    lens, shared, page, Hq, Hkv, D, kv = case
    note(f"precision of decode {len(lens)}x{max(lens)} shared {shared} of {page} {Hq}/{Hkv} x {D} {kv}")
    q, k, v, table, lens = decode_make(sum(lens) + D, lens, shared, page, Hq, Hkv, D, kv)
    got = decode_call(dev(q), dev(k), dev(v), table, lens, shared_pages=shared)
    mine, plain, g = [], [], Hq // Hkv
    for b in range(len(lens)):
        n = int(lens[b])
        for j in sorted({0, Hkv - 1}):
            kk, vv = (ref.gather(x, table[b], n)[:, j] for x in (k, v))
            hs = slice(j * g, j * g + g)
            e = ap.errors(got[b, hs], q[b, hs], kk, vv, [n] * g, D ** -0.5)
            mine.append(e[0])
            plain.append(e[1])
    grade(ap.rms(mine), ap.rms(plain), "all rows")
