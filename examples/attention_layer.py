"""One attention layer served from a paged cache: a prompt, several samples of
it, and their next tokens.

    python examples/attention_layer.py

The prompt's tokens go through the QKV projection, the rotary packing, causal
attention and the output projection, and their K and V into the cache.  The
sequence is then forked: the samples share the prompt's whole pages and get a
copy of the last, partly filled one.  Each step projects one token per sample,
reserves and writes its place in the cache, and attends to the prompt's pages
(read once for all samples) and its own.  In the end the samples' pages are
given up and the pool is made dense.

``run`` returns the largest error of every output against the same layer in
FP64, relative to the largest value.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import compensated_fp32_projection_amd as cf  # noqa: E402


class Layer:
    """QKV projection, rotary packing, attention, output projection; weights FP16 [in, out]."""

    def __init__(self, heads, dim, generator):
        self.heads, self.dim, width = heads, dim, heads * dim
        self.w_qkv, self.w_out = (
            (torch.randn(width, n, generator=generator, device="cuda") / width ** 0.5).half() for n in (3 * width, width))

    def project(self, x, positions):
        """q, k, v as [tokens, heads, dim]."""
        return [t.transpose(0, 1) for t in cf.qkv_rotary(cf.linear(x, self.w_qkv), self.heads, self.dim, positions)]

    def finish(self, o):
        return cf.linear(o.reshape(o.shape[0], -1), self.w_out)


class Cache:
    """Pools of pages, their counts, and the tables and lengths of the running sequences."""

    def __init__(self, pages, heads, page, dim, width, dtype):
        self.k, self.v = (torch.zeros(pages, heads, page, dim, dtype=dtype, device="cuda") for _ in range(2))
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
        self.table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.page = page

    def append(self, k, v, cu):
        self.table, self.refs = cf.cache_reserve(self.table, self.lens, self.refs, cu, self.page)
        self.lens = cf.cache_append(k, v, cu, self.k, self.v, self.table, self.lens)

    def fork(self, parents):
        """Children of the running sequences, which give up their own pages."""
        old = self.table
        self.table, self.refs, self.lens = cf.cache_fork(self.k, self.v, old, self.lens, self.refs, parents)
        self.refs = cf.cache_free(old, self.refs)

    def keep(self, rows):
        """Ends the sequences that are not in `rows`, and makes the pool dense."""
        gone = torch.ones(self.table.shape[0], dtype=torch.bool, device="cuda")
        gone[rows] = False
        self.refs = cf.cache_free(self.table[gone], self.refs)
        self.table, self.refs, live = cf.cache_compact(self.k, self.v, self.table[rows], self.refs)
        self.lens = self.lens[rows]
        return live


def reference(layer, q, k, v, dtype):
    """The output projection of attention of q [n, heads, dim] at the end of keys k, v, in FP64."""
    q, k, v = q.double(), k.to(dtype).double(), v.to(dtype).double()
    e = torch.einsum("nhd,mhd->hnm", q, k) * layer.dim ** -0.5
    n, m = q.shape[0], k.shape[0]
    later = torch.arange(m, device="cuda")[None] > torch.arange(n, device="cuda")[:, None] + m - n
    o = torch.einsum("hnm,mhd->nhd", e.masked_fill(later, float("-inf")).softmax(-1), v)
    return o.reshape(n, -1) @ layer.w_out.double()


def run(tokens=200, samples=6, steps=5, heads=12, dim=64, page=16, dtype=torch.float32, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    layer = Layer(heads, dim, g)
    width = -(-(tokens + steps) // page)
    cache = Cache(width * (samples + 1), heads, page, dim, width, dtype)
    off = []

    def compare(got, want):
        off.append(float((got.double() - want).abs().max() / want.abs().max()))

    x = torch.randn(tokens, heads * dim, generator=g, device="cuda")
    cu = torch.tensor([0, tokens], dtype=torch.int32, device="cuda")
    q, k, v = layer.project(x, torch.arange(tokens, device="cuda"))
    compare(layer.finish(cf.attention_prompt(q, k, v, cu)), reference(layer, q, k, v, torch.float32))
    cache.append(k, v, cu)

    cache.fork(torch.zeros(samples, dtype=torch.int32, device="cuda"))
    seen_k, seen_v = [k] * samples, [v] * samples
    each = torch.arange(samples + 1, dtype=torch.int32, device="cuda")
    for _ in range(steps):
        x = torch.randn(samples, heads * dim, generator=g, device="cuda")
        q, k, v = layer.project(x, cache.lens.long())
        cache.append(k, v, each)
        o = cf.attention_decode(q, cache.k, cache.v, cache.table, cache.lens, shared_pages=tokens // page)
        got = layer.finish(o)
        for i in range(samples):
            seen_k[i], seen_v[i] = torch.cat([seen_k[i], k[i:i + 1]]), torch.cat([seen_v[i], v[i:i + 1]])
            compare(got[i:i + 1], reference(layer, q[i:i + 1], seen_k[i], seen_v[i], dtype))

    # Half of the samples end; the others go on from the dense pool.
    rows = torch.arange(0, samples, 2, device="cuda")
    live = cache.keep(rows)
    q = torch.randn(len(rows), heads, dim, generator=g, device="cuda")
    got = layer.finish(cf.attention_decode(q, cache.k, cache.v, cache.table, cache.lens, shared_pages=tokens // page))
    for j, i in enumerate(rows.tolist()):
        compare(got[j:j + 1], reference(layer, q[j:j + 1], seen_k[i], seen_v[i], dtype))
    assert int(live) == int((cache.refs > 0).sum()) and bool((cache.refs[int(live):] == 0).all())
    return max(off)


if __name__ == "__main__":
    for dtype in (torch.float32, torch.float16):
        print(f"{dtype} cache: largest error {run(dtype=dtype):.2g} of the largest value")
