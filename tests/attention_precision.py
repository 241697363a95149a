"""The error of attention results beside that of plain FP32 arithmetic.

``errors`` gives the RMS error of rows against the definition in FP64, relative
to sum w |v| / sum w of each output, and that of the same rows in plain FP32
(numpy: products and sums in FP32, blocked as BLAS blocks them).

An FP32-grade result may be RATIO times the plain form's.  Operands in two FP16
parts keep 22 bits: an element is off by up to 2^-22, 2^-23.8 in the mean square,
and so are the dropped products of two low parts; for a score's two operands
together 2^-23 of the norm of its products, where plain FP32 has 2^-25 (the
rounding of each sum) or more: a factor of 4 at most.  Weights and values give
the same once more, and sums in the order of the keys instead of BLAS' blocks
a factor of up to 2: 8 in all.  One part instead of two (2^-11 an element)
is some 2^10 times plain FP32's.
"""
import numpy as np

RATIO = 8.0


def rms(x):
    return float(np.sqrt(np.mean(np.square(x))))


def plain(q, k, v, limits, scale, cut=lambda name, x: x):
    """Rows in FP32; ``cut`` may coarsen an operand ("q", "k", "v" or "w") on its way."""
    f = np.float32
    s = (cut("q", q.astype(f)) @ cut("k", k.astype(f)).T) * f(scale)
    s[np.arange(k.shape[0])[None] >= np.asarray(limits)[:, None]] = -np.inf
    w = np.exp(s - s.max(axis=1, keepdims=True))
    return (cut("w", w) @ cut("v", v.astype(f))) / w.sum(axis=1, keepdims=True)


def exact(q, k, v, limits, scale):
    """(out, sum w |v| / sum w) in FP64."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    s = (q @ k.T) * scale
    s[np.arange(k.shape[0])[None] >= np.asarray(limits)[:, None]] = -np.inf
    w = np.exp(s - s.max(axis=1, keepdims=True))
    w /= w.sum(axis=1, keepdims=True)
    return w @ v, w @ np.abs(v)


def errors(got, q, k, v, limits, scale):
    want, norm = exact(q, k, v, limits, scale)
    return rms((got - want) / norm), rms((plain(q, k, v, limits, scale) - want) / norm)
