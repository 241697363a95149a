"""Beam search over an 8-bit cache: prompts in two pieces, then steps of several
beams to a prompt.

    python examples/beam_search.py

One attention layer with grouped heads between an embedding and a vocabulary
projection, random weights.  A prompt's first piece goes through the projection,
rotary positions and causal attention; its K and V are written into the cache in
8 bits.  The second piece attends to what the cache holds of the first, read
back.  Then the prompts' best continuations become their beams: the sequences
fork (whole pages are shared), and each step turns, writes and attends to one
token of every beam, selects the best continuations over beams and vocabulary,
and puts histories and pages in the beams' new order.

``run`` returns the beams' tokens and scores and the largest error, relative to
the largest value, of every attention result against FP64 on the values that the
cache stands for.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import compensated_fp32_projection_amd as cf  # noqa: E402


class Model:
    """Embedding, QKV projection with grouped heads, rotary positions, output and vocabulary projections."""

    def __init__(self, vocab, width, heads, kv_heads, dim, generator):
        def weights(*shape):
            return torch.randn(*shape, generator=generator, device="cuda") / shape[0] ** 0.5

        self.heads, self.kv_heads, self.dim = heads, kv_heads, dim
        self.embed = weights(vocab, width) * vocab ** 0.5
        self.w_qkv = weights(width, (heads + 2 * kv_heads) * dim).half()
        self.w_out, self.w_vocab = weights(heads * dim, width).half(), weights(width, vocab).half()
        # Twice as long a context as trained.
        self.frequencies, self.amplitude = cf.rotary_frequencies(dim, scaling="parts", factor=2.0, trained=512)

    def project(self, tokens, positions):
        """(x, q, k, v) of tokens at their positions; q, k, v [tokens, heads, dim], views of the projection's rows."""
        x = self.embed[tokens.long()]
        y = cf.linear(x, self.w_qkv).view(len(tokens), -1, self.dim)
        q, k, v = y.split([self.heads, self.kv_heads, self.kv_heads], dim=1)
        cf.rotary(q, k, self.frequencies, positions, amplitude=self.amplitude, q_out=q, k_out=k)
        return x, q, k, v

    def logits(self, x, o):
        return cf.linear(x + cf.linear(o.reshape(len(x), -1), self.w_out), self.w_vocab)


class Cache:
    """The 8-bit pools, their pages' counts, and the tables and lengths of the running sequences."""

    def __init__(self, sequences, pages, model, page, block, width, dtype):
        self.pools = cf.Cache8.empty(pages, model.kv_heads, page, model.dim, block=block, dtype=dtype)
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.table = torch.full((sequences, width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(sequences, dtype=torch.int32, device="cuda")
        self.page = page

    def append(self, k, v, cu):
        self.table, self.refs = cf.cache_reserve(self.table, self.lens, self.refs, cu, self.page)
        self.lens = cf.cache8_append(k, v, cu, self.pools, self.table, self.lens)

    def read(self):
        """(k, v, cu) of all tokens, packed."""
        cu = starts(self.lens)
        return (*cf.cache8_read(self.pools, self.table, cu, int(cu[-1])), cu)

    def reorder(self, parents):
        old = self.table
        self.table, self.refs, self.lens = cf.cache8_fork(self.pools, old, self.lens, self.refs, parents)
        self.refs = cf.cache_free(old, self.refs)


def starts(lens):
    return torch.nn.functional.pad(lens.cumsum(0), (1, 0)).to(torch.int32)


def reference(q, k, v, causal_rows):
    """Attention of q [n, heads, dim] over k, v [m, kv heads, dim] in FP64; row i sees the first m - n + 1 + i of them."""
    g = q.shape[1] // k.shape[1]
    q, k, v = q.double(), k.double().repeat_interleave(g, 1), v.double().repeat_interleave(g, 1)
    e = torch.einsum("nhd,mhd->hnm", q, k) * q.shape[2] ** -0.5
    n, m = q.shape[0], k.shape[0]
    later = torch.arange(m, device="cuda")[None] > torch.arange(n, device="cuda")[:, None] + m - n
    return torch.einsum("hnm,mhd->nhd", (e.masked_fill(later, float("-inf")) if causal_rows else e).softmax(-1), v)


def run(prompts=(70, 33, 101), beams=4, steps=12, vocab=1000, width=256, heads=8, kv_heads=2, dim=64, page=16, block=8,
        dtype=torch.int8, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    model = Model(vocab, width, heads, kv_heads, dim, g)
    S = len(prompts)
    longest = max(prompts) + steps + 1
    wide = -(-longest // page)
    cache = Cache(S, 3 * S * beams * wide + S, model, page, block, wide, dtype)
    off = []

    def compare(got, want):
        off.append(float((got.double() - want).abs().max() / want.abs().max()))

    # The prompts, in two pieces of about half each.
    last = None
    for piece in range(2):
        n = torch.tensor([(p + 1) // 2 if piece == 0 else p // 2 for p in prompts], dtype=torch.int32, device="cuda")
        cu, counts = starts(n), n.tolist()
        tokens = torch.randint(0, vocab, (sum(counts),), generator=g, device="cuda")
        before = cache.lens.tolist()
        positions = torch.cat([torch.arange(b, b + c, device="cuda") for b, c in zip(before, counts)])
        x, q, k, v = model.project(tokens, positions)
        cache.append(k, v, cu)
        keys, values, cu_k = cache.read()
        o = cf.attention_prompt(q, keys, values, cu, cu_k)
        for i in range(S):
            a, b, a2, b2 = cu[i], cu[i + 1], cu_k[i], cu_k[i + 1]
            compare(o[a:b], reference(q[a:b], keys[a2:b2], values[a2:b2], True))
        last = (cu[1:] - 1).long()
        logits = model.logits(x[last], o[last])

    # Each prompt's best continuations are its beams.
    scores = torch.zeros(S, 1, device="cuda")
    history = torch.zeros(S, 0, dtype=torch.int32, device="cuda")
    done, eos = None, 0
    for step in range(steps):
        parents, tokens, scores, done = cf.beam_select(logits, scores, n=beams, done=done, eos=eos)
        rows = parents.flatten()
        history = torch.cat([cf.beam_reorder(history, rows), tokens.reshape(-1, 1)], dim=1)
        cache.reorder(rows)
        if step == steps - 1 or bool(done.all()):
            break
        x, q, k, v = model.project(tokens.flatten(), cache.lens.long())
        cache.append(k, v, torch.arange(S * beams + 1, dtype=torch.int32, device="cuda"))
        o = cf.attention8_decode(q, cache.pools, cache.table, cache.lens)
        keys, values, cu_k = cache.read()
        for i in range(S * beams):
            a, b = cu_k[i], cu_k[i + 1]
            compare(o[i:i + 1], reference(q[i:i + 1], keys[a:b], values[a:b], False))
        logits = model.logits(x, o)
    return history.reshape(S, beams, -1), scores, max(off)


if __name__ == "__main__":
    for dtype in (torch.int8, torch.float8_e4m3fn):
        history, scores, off = run(dtype=dtype)
        print(f"{dtype} cache: best of each prompt {history[:, 0].tolist()}, scores {scores[:, 0].tolist()}, largest "
              f"attention error {off:.2g} of the largest value")
