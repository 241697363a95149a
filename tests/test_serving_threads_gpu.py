"""Rotary, 8-bit cache and beam calls in flight together: on different streams,
and from several host threads on one stream that share its workspace, the bits
that each call gives alone."""
import threading

import numpy as np
import pytest
import torch

import compensated_fp32_projection_amd as cf
from gpu_helpers import note
from test_attention8_gpu import problem
from test_cache8_gpu import cache_of, dev

pytestmark = pytest.mark.gpu


class Decode:
    def __init__(self, seed, lens, Hq, Hkv, D, page, block, kind):
        q, arrays, table, lens = problem(np.random.default_rng(seed), lens, Hq, Hkv, D, page, block, kind)
        self.cache = cache_of(arrays, kind)[0]
        self.args = dev(q), self.cache, dev(table), dev(lens)

    def run(self, **kw):
        return [cf.attention8_decode(*self.args, **kw)]


class Beams:
    def __init__(self, seed, S, beams, V, n):
        rng = np.random.default_rng(seed)
        self.x, self.n = dev((rng.standard_normal((S * beams, V)) * 3).astype(np.float32)), n
        self.scores = dev((-20 * rng.random((S, beams))).astype(np.float32))
        self.states = dev(rng.integers(0, 1000, (S * beams, 77)).astype(np.int32))

    def run(self, **kw):
        r = cf.beam_select(self.x, self.scores, n=self.n, **kw)
        return [*r, cf.beam_reorder(self.states, r[0], stream=kw.get("stream"))]


class Turns:
    def __init__(self, seed, T, Hq, Hkv, D):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.q, self.k = (torch.randn(T, h, D, generator=g, device="cuda") for h in (Hq, Hkv))
        self.f = cf.rotary_frequencies(D)[0]

    def run(self, **kw):
        return list(cf.rotary(self.q, self.k, self.f, stream=kw.get("stream")))


class Reads:
    def __init__(self, seed, lens, kind):
        _, arrays, table, lens = problem(np.random.default_rng(seed), lens, 2, 2, 64, 16, 8, kind)
        self.cache, self.table, self.n = cache_of(arrays, kind)[0], dev(table), int(lens.sum())
        self.cu = dev(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32))

    def run(self, **kw):
        return list(cf.cache8_read(self.cache, self.table, self.cu, self.n, stream=kw.get("stream")))


class Pages:
    """Children of some sequences, and the pool made dense (pages of zeros: the same pool after any number of runs)."""

    def __init__(self, seed, P):
        rng = np.random.default_rng(seed)
        W = 6
        S = P // (2 * W)
        self.cache = cf.Cache8.empty(P, 2, 16, 64, block=8)
        self.table = dev(rng.permutation(P)[:S * W].reshape(S, W).astype(np.int32))
        self.lens = dev(rng.integers(1, W * 16, S).astype(np.int32))
        refs = np.zeros(P, np.int32)
        refs[self.table.cpu().numpy()] = 1
        self.refs = dev(refs)
        self.parents = dev(rng.integers(0, S, S // 2).astype(np.int32))

    def run(self, **kw):
        return [*cf.cache8_fork(self.cache, self.table, self.lens, self.refs, self.parents, **kw),
                *cf.cache8_compact(self.cache, self.table, self.refs, **kw)]


def jobs():
    return [Decode(1, [9000, 4000], 8, 2, 128, 64, 64, "i8"), Beams(2, 3, 4, 20000, 4), Turns(3, 900, 8, 2, 128), Pages(4, 600),
            Decode(5, [700] * 30, 6, 6, 64, 16, 4, "e4m3"), Beams(6, 20, 8, 5000, 8), Reads(7, [500, 3, 900], "i8"), Pages(8, 3000),
            Decode(9, [3000], 16, 1, 72, 4, 1, "i8"), Reads(10, [64] * 20, "e4m3")]


def same(got, want, what):
    for g, w in zip(got, want):
        assert torch.equal(g, w), what


def test_many_streams():
    work = jobs()
    note("serving jobs alone")
    want = [j.run() for j in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    note(f"serving jobs on {len(work)} streams")
    got = [[j.run(stream=s) for j, s in zip(work, streams)] for _ in range(3)]
    torch.cuda.synchronize()
    for r in got:
        for i, (g, w) in enumerate(zip(r, want)):
            same(g, w, f"job {i}")


def test_threads_on_one_stream():
    """The helpers' native form in one thread and their Python form in others."""
    work = jobs()
    note("serving jobs alone")
    want = [j.run() for j in work]
    torch.cuda.synchronize()
    results, errors = [[], [], []], []

    def loop(n):
        try:
            stream = torch.cuda.current_stream()
            for r in range(4):
                for i in range(len(work)):
                    k = (i + 3 * n) % len(work)
                    if not isinstance(work[k], Pages) or n == 1:  # (two runs of one pool's would write it at once)
                        results[n].append((k, work[k].run() if n == 0 else work[k].run(stream=stream)))
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    note("serving jobs of three threads on one stream")
    threads = [threading.Thread(target=loop, args=(n,)) for n in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for n, done in enumerate(results):
        for k, got in done:
            same(got, want[k], f"thread {n} job {k}")


def test_a_step_captured_into_a_graph():
    """Turned, written, attended to, selected, reordered and forked in one graph: every replay on new inputs, with eager
    work between them, is the eager calls' result."""
    S, beams, H, D, V, page = 3, 4, 2, 64, 3001, 16
    rows, W, P = S * beams, 6, 200
    rng = np.random.default_rng(11)
    f, a = cf.rotary_frequencies(D, scaling="linear", factor=2.0)
    q, k, v = (torch.randn(rows, h, D, device="cuda") for h in (8, H, H))
    logits, scores = torch.randn(rows, V, device="cuda"), torch.zeros(S, beams, device="cuda")
    start_lens = rng.integers(1, 60, rows).astype(np.int32)
    start_table = np.full((rows, W), -1, np.int32)
    ids = rng.permutation(P)
    at = 0
    for s in range(rows):
        n = -(-(int(start_lens[s]) + 1) // page)
        start_table[s, :n] = ids[at:at + n]
        at += n
    start_refs = np.zeros(P, np.int32)
    start_refs[start_table[start_table >= 0]] = 1
    table, lens, refs = dev(start_table), dev(start_lens), dev(start_refs)
    each = torch.arange(rows + 1, dtype=torch.int32, device="cuda")
    pools = cf.Cache8.empty(P, H, page, D, block=8)
    first = [t.clone() for t in (pools.k, pools.v)]
    for t in (pools.k_scales, pools.v_scales):
        t.fill_(2.0 ** -6)

    def step(ws, stream=None):
        qt, kt = cf.rotary(q, k, f, lens.long(), amplitude=a, stream=stream)
        n = cf.cache8_append(kt, v, each, pools, table, lens, stream=stream)
        o = cf.attention8_decode(qt, pools, table, n, workspace=ws, stream=stream)
        r = cf.beam_select(logits, scores, workspace=ws, stream=stream)
        o = cf.beam_reorder(o, r[0], stream=stream)
        forked = cf.cache8_fork(pools, table, n, refs, r[0].flatten(), workspace=ws, stream=stream)
        return [o, *r, *forked]

    def reset():
        pools.k.copy_(first[0])
        pools.v.copy_(first[1])
        pools.k_scales.fill_(2.0 ** -6)
        pools.v_scales.fill_(2.0 ** -6)

    note("serving step captured")
    ws = cf.Workspace()
    step(ws)
    reset()
    torch.cuda.synchronize()
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(st):
        with torch.cuda.graph(g, stream=st):
            outs = step(ws, st)
    torch.cuda.synchronize()
    for i in range(4):
        for t in (q, k, v, logits):
            t.normal_()
        scores.uniform_(-5, 0)
        reset()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*outs, pools.k, pools.v, pools.k_scales, pools.v_scales)]
        reset()
        want = [*step(cf.Workspace()), pools.k, pools.v, pools.k_scales, pools.v_scales]
        torch.cuda.synchronize()
        same(got, want, f"replay {i}")
