"""The 8-bit cache from its definition, in numpy: one block of one head at a time."""
import numpy as np

TOP = {"i8": 127.0, "e4m3": 448.0}
LEAST = 2.0 ** -126

# Every float code's value; 0x7F and 0xFF count as 480.
_E4M3 = np.zeros(256)
for _c in range(256):
    _e, _m = (_c >> 3) & 15, _c & 7
    _v = _m * 2.0 ** -9 if _e == 0 else (8 + _m) * 2.0 ** (_e - 10)
    _E4M3[_c] = -_v if _c & 128 else _v


def values(codes, kind):
    """Values of codes given as bytes (uint8)."""
    return codes.view(np.int8).astype(np.float64) if kind == "i8" else _E4M3[codes]


def nearest(y, kind):
    """Codes (bytes) of y (exact quotients, FP64), to nearest even."""
    if kind == "i8":
        return np.rint(y).astype(np.int8).view(np.uint8)
    size = np.maximum(np.abs(y), 2.0 ** -6)
    step = 2.0 ** (np.floor(np.log2(size)) - 3)
    r = np.rint(y / step) * step
    a = np.abs(r)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    code = np.where(a < 2.0 ** -6, a * 512, (e + 7) * 8 + a / 2.0 ** e * 8 - 8).astype(np.uint8)
    return code | np.where(np.signbit(y), 128, 0).astype(np.uint8)


def fresh_scale(most, kind):
    if kind == "i8":
        return max(float(np.float32(most) * (np.float32(1) / np.float32(127))), LEAST)
    s = LEAST
    while most > 448 * s:
        s *= 2
    return s


def append(codes, scales, x, cu, lens, table, block, kind):
    """Writes x [T, H, D] into codes [P, H, page, D] (bytes) and scales [P, H, blocks], in place."""
    P, H, page, D = codes.shape
    for s in range(len(lens)):
        n = int(cu[s + 1]) - int(cu[s])
        if lens[s] < 0:
            continue
        ln = int(lens[s])
        for p0 in range(ln // block * block, ln + n, block):
            a, b = max(p0, ln), min(p0 + block, ln + n)
            entry = p0 // page
            if a >= b or entry >= table.shape[1] or not 0 <= table[s, entry] < P:
                continue
            p, o = table[s, entry], p0 % page
            for h in range(H):
                new = x[cu[s] + a - ln:cu[s] + b - ln, h].astype(np.float64)
                most = np.abs(new).max()
                old = float(scales[p, h, o // block])
                if not np.isfinite(new).all():
                    scale = np.nan
                elif p0 >= ln:
                    scale = fresh_scale(most, kind)
                elif not (LEAST <= old < np.inf):
                    scale = np.nan
                else:
                    scale = old
                    while most > float(np.float32(old) * np.float32(TOP[kind])) * (scale / old):
                        scale *= 2
                    if scale != old:
                        there = codes[p, h, o:o + ln - p0]
                        codes[p, h, o:o + ln - p0] = nearest(values(there, kind) * (old / scale), kind)
                scales[p, h, o // block] = scale
                codes[p, h, o + a - p0:o + b - p0] = 0 if np.isnan(scale) else nearest(new / scale, kind)


def read(codes, scales, cu, first, table, block, kind, out, dtype):
    """Fills out [T, H, D]; c s rounded to FP32, then to dtype."""
    P, H, page, D = codes.shape
    for s in range(len(cu) - 1):
        for t in range(max(cu[s], 0), min(cu[s + 1], len(out))):
            pos = (int(first[s]) if first is not None else 0) + t - int(cu[s])
            entry = pos // page
            if pos < 0 or entry >= table.shape[1] or not 0 <= table[s, entry] < P:
                out[t] = np.nan
                continue
            p, o = table[s, entry], pos % page
            with np.errstate(over="ignore"):
                out[t] = (values(codes[p, :, o], kind).astype(np.float32) *
                          scales[p, :, o // block][:, None].astype(np.float32)).astype(dtype)
    return out
