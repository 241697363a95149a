"""Attention and cache calls in flight together: on different streams, and from
several host threads on one stream that share its workspace, the bits that each
call gives alone."""
import threading

import numpy as np
import pytest
import torch

import compensated_fp32_projection_amd as cf
from gpu_helpers import note
from test_attention_decode_gpu import make as decode_make
from test_attention_prompt_gpu import dev, make, starts

pytestmark = pytest.mark.gpu


class Prompt:
    def __init__(self, seed, lens, Hq, Hkv, D, kv):
        self.args = [dev(x) for x in make(seed, lens, lens, Hq, Hkv, D, kv)] + [dev(starts(lens))]

    def run(self, **kw):
        return [cf.attention_prompt(*self.args, **kw)]


class Decode:
    def __init__(self, seed, lens, shared, page, Hq, Hkv, D, kv):
        self.args = [dev(x) for x in decode_make(seed, lens, shared, page, Hq, Hkv, D, kv, unused=0)]
        self.shared = shared

    def run(self, **kw):
        return [cf.attention_decode(*self.args, shared_pages=self.shared, **kw)]


class Pages:
    """Children of some sequences, and the pool made dense (pages of zeros: the same pool after any number of runs)."""

    def __init__(self, seed, P):
        rng = np.random.default_rng(seed)
        W = 6
        S = P // (2 * W)
        self.pools = [torch.zeros(P, 2, 16, 64, dtype=torch.float16, device="cuda") for _ in range(2)]
        self.table = dev(rng.permutation(P)[:S * W].reshape(S, W).astype(np.int32))
        self.lens = dev(rng.integers(1, W * 16, S).astype(np.int32))
        refs = np.zeros(P, np.int32)
        refs[self.table.cpu().numpy()] = 1
        self.refs = dev(refs)
        self.parents = dev(rng.integers(0, S, S // 2).astype(np.int32))

    def run(self, **kw):
        return [*cf.cache_fork(*self.pools, self.table, self.lens, self.refs, self.parents, **kw),
                *cf.cache_compact(*self.pools, self.table, self.refs, **kw)]


def jobs():
    return [Prompt(71, [1100], 12, 12, 64, "f32"), Decode(72, [2000, 1990], 0, 16, 4, 1, 64, "f32"), Pages(73, 600),
            Prompt(74, [290, 310, 270], 32, 8, 128, "f32"), Decode(75, [6200] * 20, 90, 64, 64, 8, 128, "f16"),
            Prompt(76, [300], 4, 2, 64, "f16"), Pages(77, 3000), Prompt(78, [1500], 12, 12, 64, "f32")]


def same(got, want, what):
    for g, w in zip(got, want):
        assert torch.equal(g, w), what


def test_many_streams():
    work = jobs()
    note("attention jobs alone")
    want = [j.run() for j in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    note(f"attention jobs on {len(work)} streams")
    got = [[j.run(stream=s) for j, s in zip(work, streams)] for _ in range(3)]
    torch.cuda.synchronize()
    for r in got:
        for i, (g, w) in enumerate(zip(r, want)):
            same(g, w, f"job {i}")


def test_threads_on_one_stream():
    """The helpers' native form in one thread and their Python form in others."""
    work = jobs()
    note("attention jobs alone")
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

    note("attention jobs of three threads on one stream")
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
