"""The attention and cache operators from their definitions, in numpy.

Attention is in FP64, with a bound on what an FP32-grade evaluation may be
off.  With e = 2^-24 (half a step of FP32), for row i:

  * a score s = scale * sum_d q_d k_d formed from parts with 22 significant
    bits (an error of 2^-22 of each product for each operand's split, plus
    the dropped product of the two low parts) and summed in FP32 is off by at
    most ds = scale * sum_d |q_d k_d| * (D + 16) e: D additions and 12 e for
    the two splits and the dropped product, 4 e for scaling;
  * a weight exp(s - m) is then off by a relative 2 ds (its own score's and
    the maximum's error) and 8 e (the exponential and its argument's
    rounding at |s - m| < 100 is a further 100 e * log2 e, counted with the
    scores' magnitude below);
  * weights are split into parts of 22 bits (4 e), and sums of n terms are
    off by n e: numerator and denominator together 2 (n + 8) e.

  |o - o64| <= [4 max_j ds_j + (2 n + 64 + 2 * 1.5 max_j |s_j - m|) e] * sum_j w_j |v_j| / sum_j w_j.
"""
import numpy as np

E = 2.0 ** -24


def attend(q, k, v, limits, scale):
    """(out, bound) of rows q [R, D] over keys k, v [n, D], row i seeing the first limits[i]."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    R, D = q.shape
    out, bound = np.zeros((R, D)), np.zeros((R, D))
    for i in range(R):
        n = int(limits[i])
        if n <= 0:
            continue
        s = scale * (k[:n] @ q[i])
        ds = abs(scale) * (np.abs(k[:n]) @ np.abs(q[i])) * (D + 16) * E
        w = np.exp(s - s.max())
        out[i] = (w @ v[:n]) / w.sum()
        seen = w > 1e-30
        spread = min(100.0, (s.max() - s[seen]).max())
        rel = 4 * ds[seen].max() + (2 * n + 64 + 3 * spread) * E
        bound[i] = rel * (w @ np.abs(v[:n])) / w.sum()
    return out, bound


def prompt(q, k, v, cu_q, cu_k, causal=True, scale=None):
    """(out, bound, rows written) of packed prompts: q [Tq, Hq, D], k and v [Tk, Hkv, D]."""
    Tq, Hq, D = q.shape
    g = Hq // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out, bound, written = np.zeros((Tq, Hq, D)), np.zeros((Tq, Hq, D)), np.zeros(Tq, bool)
    for s in range(len(cu_q) - 1):
        a, b, a2, b2 = cu_q[s], cu_q[s + 1], cu_k[s], cu_k[s + 1]
        lq, lk = b - a, b2 - a2
        limits = np.clip(np.arange(lq) + lk - lq + 1, 0, lk) if causal else np.full(lq, lk)
        written[a:b] = True
        for h in range(Hq):
            out[a:b, h], bound[a:b, h] = attend(q[a:b, h], k[a2:b2, h // g], v[a2:b2, h // g], limits, scale)
    return out, bound, written


def gather(pages, row, n):
    """The first n tokens [n, Hkv, D] of the pages [P, Hkv, page, D] a table row names."""
    page = pages.shape[2]
    ids = np.asarray(row[:-(-n // page)], np.int64)
    return pages[ids].transpose(0, 2, 1, 3).reshape(-1, pages.shape[1], pages.shape[3])[:n]


def decode(q, k_pages, v_pages, table, lens, scale=None):
    B, Hq, D = q.shape
    g = Hq // k_pages.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out, bound = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    for b in range(B):
        n = int(lens[b])
        k, v = gather(k_pages, table[b], n), gather(v_pages, table[b], n)
        for h in range(Hq):
            o, e = attend(q[b, h:h + 1], k[:, h // g], v[:, h // g], [n], scale)
            out[b, h], bound[b, h] = o[0], e[0]
    return out, bound


# -- the cache's bookkeeping ------------------------------------------------------

def free_pages(refs):
    return [p for p, r in enumerate(refs) if r <= 0]


def reserve(table, lens, refs, cu, page):
    table, refs = table.copy(), refs.copy()
    free, missing = free_pages(refs), 0
    for s in range(table.shape[0]):
        need = max(0, -(-(int(lens[s]) + int(cu[s + 1]) - int(cu[s])) // page))
        missing += max(0, need - table.shape[1])
        for j in range(min(need, table.shape[1])):
            if table[s, j] < 0:
                if free:
                    table[s, j] = free.pop(0)
                    refs[table[s, j]] = 1
                else:
                    missing += 1
    return table, refs, missing


def append(k, v, cu, k_pages, v_pages, table, lens):
    P, _, page, _ = k_pages.shape
    for s in range(table.shape[0]):
        for i, t in enumerate(range(cu[s], cu[s + 1])):
            pos = int(lens[s]) + i
            if pos < 0 or pos // page >= table.shape[1]:
                continue
            p = table[s, pos // page]
            if 0 <= p < P:
                k_pages[p, :, pos % page] = k[t].astype(k_pages.dtype)
                v_pages[p, :, pos % page] = v[t].astype(v_pages.dtype)
    return lens + np.diff(cu).astype(np.int32)


def fork(k_pages, v_pages, table, lens, refs, parents):
    P, _, page, _ = k_pages.shape
    W = table.shape[1]
    out = np.full((len(parents), W), -1, np.int32)
    out_lens, refs2 = np.zeros(len(parents), np.int32), refs.copy()
    free, missing = free_pages(refs), 0
    for c, p in enumerate(parents):
        if not 0 <= p < table.shape[0]:
            continue
        n = min(max(int(lens[p]), 0), W * page)
        whole = n // page
        out_lens[c] = whole * page
        out[c, :whole] = table[p, :whole]
        for e in out[c, :whole]:
            if 0 <= e < P:
                refs2[e] += 1
        if n % page and 0 <= table[p, whole] < P:
            if free:
                out[c, whole] = free.pop(0)
                refs2[out[c, whole]] = 1
                k_pages[out[c, whole]] = k_pages[table[p, whole]]
                v_pages[out[c, whole]] = v_pages[table[p, whole]]
                out_lens[c] = n
            else:
                missing += 1
    return out, refs2, out_lens, missing


def free(rows, refs):
    refs = refs.copy()
    for e in rows.ravel():
        if 0 <= e < len(refs):
            refs[e] -= 1
    return refs


def compact(k_pages, v_pages, table, refs):
    n = int((refs > 0).sum())
    src = [p for p in range(n, len(refs)) if refs[p] > 0]
    dst = [p for p in range(n) if refs[p] <= 0]
    refs, to = refs.copy(), np.arange(len(refs))
    for a, b in zip(src, dst):
        k_pages[b], v_pages[b], refs[b], to[a] = k_pages[a], v_pages[a], refs[a], b
    refs[n:] = 0
    named = (table >= 0) & (table < len(refs))
    return np.where(named, to[np.where(named, table, 0)], table).astype(np.int32), refs, n
