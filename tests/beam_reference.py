"""A step of beam search from its definition, in numpy and FP64."""
import numpy as np


def offers(logits, score, done, eos):
    """(totals, tokens) of a beam's offers, in order."""
    if not np.isfinite(score):
        return np.zeros(0), np.zeros(0, int)
    if done:
        return np.array([np.float64(score)]), np.array([eos])
    x = logits.astype(np.float64)
    if np.isnan(x).any() or not -np.inf < x.max() < np.inf:
        return np.zeros(0), np.zeros(0, int)
    lse = x.max() + np.log(np.exp(x - x.max()).sum())
    order = np.lexsort((np.arange(len(x)), -x))
    order = order[x[order] > -np.inf]
    return np.float64(score) + (x[order] - lse), order


def select(logits, scores, n, done=None, eos=-1):
    """(parents, tokens, scores FP64, done) and the least distance between totals of different beams that decide."""
    S, beams = scores.shape
    parents, tokens = np.full((S, n), -1, np.int32), np.full((S, n), eos, np.int32)
    out, ended, gap = np.full((S, n), -np.inf), np.ones((S, n), bool), np.inf
    for s in range(S):
        rows = []
        for b in range(beams):
            was = done is not None and bool(done[s, b])
            total, token = offers(logits[s * beams + b], scores[s, b], was, eos)
            rows += [(-v, b, i, t, was) for i, (v, t) in enumerate(zip(total[:n + 1], token[:n + 1]))]
        rows.sort(key=lambda r: r[:3])
        for i, (v, b, _, t, was) in enumerate(rows[:n]):
            parents[s, i], tokens[s, i], out[s, i] = s * beams + b, t, -v
            ended[s, i] = was or (eos >= 0 and t == eos)
        for p, q in zip(rows[:n], rows[1:n + 1]):
            if p[1] != q[1] and p[0] != q[0]:
                gap = min(gap, q[0] - p[0])
    return parents, tokens, out, ended, gap
