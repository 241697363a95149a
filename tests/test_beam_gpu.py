"""GPU tests of beam search against its definition in FP64: whole results.

Totals of different beams that decide are 2e-6 apart at least in these inputs
(asserted), or equal: the sums of 2^-22 a term, the rest FP64, put a total off by
less than 3e-7.  A score is that and one rounding to FP32 off.
"""
import numpy as np
import pytest
import torch

import beam_reference as ref
import compensated_fp32_projection_amd as cf
from gpu_helpers import note

pytestmark = pytest.mark.gpu


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check(got, want):
    torch.cuda.synchronize()
    parents, tokens, scores, done = (t.cpu().numpy() for t in got)
    assert want[4] > 2e-6, "these inputs do not decide"
    assert np.array_equal(parents, want[0]) and np.array_equal(tokens, want[1]) and np.array_equal(done, want[3])
    some = np.isfinite(want[2])
    assert np.array_equal(np.isfinite(scores), some) and (scores[~some] == -np.inf).all()
    assert (np.abs(scores[some] - want[2][some]) <= 3e-7 + np.abs(want[2][some]) * 2.0 ** -24).all()


def problem(rng, S, beams, V, spread=3.0):
    logits = (rng.standard_normal((S * beams, V)) * spread).astype(np.float32)
    scores = (-20 * rng.random((S, beams))).astype(np.float32)
    return logits, scores


@pytest.mark.parametrize("S,beams,V,n", [(1, 1, 1, 1), (1, 1, 1, 5), (2, 3, 2, 3), (1, 4, 7, 4), (3, 2, 63, 2), (1, 2, 64, 64),
                                         (2, 5, 65, 10), (1, 4, 511, 4), (2, 4, 513, 8), (1, 64, 300, 64), (5, 8, 2049, 8),
                                         (1, 4, 32003, 4), (3, 1, 50000, 64), (70, 4, 1000, 4), (2, 16, 4096, 16),
                                         (40, 8, 20001, 8), (33, 8, 32000, 5)])
def test_sizes(S, beams, V, n):
    rng = np.random.default_rng(S + V + n)
    note(f"beam {S} {beams} {V} {n}")
    logits, scores = problem(rng, S, beams, V)
    done = rng.random((S, beams)) < 0.2
    check(cf.beam_select(dev(logits), dev(scores), n=n, done=dev(done), eos=0),
          ref.select(logits, scores, n, done, 0))
    check(cf.beam_select(dev(logits), dev(scores), n=n), ref.select(logits, scores, n))


@pytest.mark.parametrize("order", ["up", "down", "equal", "blocks"])
@pytest.mark.parametrize("n", [1, 8, 64])
def test_orders(order, n):
    """Logits in order, which bring every one of them to the sort, equal ones, and runs of the largest."""
    V, S, beams = 5000, 2, 3
    x = np.arange(V) / 512.0
    if order == "down":
        x = x[::-1]
    if order == "equal":
        x = np.full(V, 0.25)
    if order == "blocks":
        x = np.where((np.arange(V) // 100) % 7 == 3, 4.0, np.arange(V) % 5)
    logits = np.stack([x + 0.5 * (b % beams) for b in range(S * beams)]).astype(np.float32)
    scores = np.array([[0, -1.5007, -3.0003], [-2, -2.0005, -0.2511]], np.float32)
    note(f"beam {order} {n}")
    check(cf.beam_select(dev(logits), dev(scores), n=n), ref.select(logits, scores, n))


@pytest.mark.parametrize("V,ld", [(1003, 1003), (1003, 1004), (2048, 2048), (997, 1200)])
def test_equal_beams_and_equal_logits(V, ld):
    """Beams that hold the same, wherever their rows lie: the lowest beam first, then the lowest token."""
    rng = np.random.default_rng(V)
    one = (rng.integers(0, 5, V) / 2).astype(np.float32)
    logits = np.zeros((8, ld), np.float32)
    logits[:, :V] = one
    scores = np.full((2, 4), -1.0, np.float32)
    note(f"beam equal {V} {ld}")
    check(cf.beam_select(dev(logits)[:, :V], dev(scores), n=10), ref.select(logits[:, :V], scores, 10))


def test_zeros_of_both_signs_are_equal():
    x = np.array([[-0.0, 0.0, -1.0, 0.0, -0.0]], np.float32)
    check(cf.beam_select(dev(x), dev(np.zeros((1, 1), np.float32)), n=5), ref.select(x, np.zeros((1, 1), np.float32), 5))


def test_masked_logits():
    """-infinity and the lowest finite value, for single tokens, whole stretches and whole rows."""
    rng = np.random.default_rng(3)
    logits, scores = problem(rng, 6, 2, 3001)
    low = np.finfo(np.float32).min
    logits[0, 1:] = -np.inf            # one token is left
    logits[1, :] = -np.inf             # none is
    logits[2, :] = low
    logits[3, :2500] = low
    logits[4, 100:] = -np.inf
    logits[5, :2999] = -np.inf
    logits[6, ::2] = low
    logits[7, 600:1200] = -np.inf
    logits[8, 3:] = -np.inf
    logits[9, 2:] = low                # two, then the lowest values
    note("beam masked")
    want = ref.select(logits, scores, 4)
    got = cf.beam_select(dev(logits), dev(scores), n=4)
    torch.cuda.synchronize()
    # The lowest value less a sum overflows FP32: such a score is -infinity, its token an offer all the same.
    check(got, (*want[:2], np.where(want[2] < low, -np.inf, want[2]), *want[3:]))


def test_what_is_no_number():
    """NaN and infinities of logits and scores: such beams offer nothing, others are as they are."""
    rng = np.random.default_rng(4)
    logits, scores = problem(rng, 4, 4, 2500)
    logits[0, 2400] = np.nan
    logits[1, 3] = np.inf
    logits[5, 77] = 3e38
    scores[1, 2], scores[1, 3], scores[2] = np.nan, np.inf, [-np.inf] * 4
    logits[12:16] = np.nan
    note("beam no numbers")
    want = ref.select(logits, scores, 4)
    assert (want[0][2:] == -1).all() and (want[0][:2] >= 0).all()
    check(cf.beam_select(dev(logits), dev(scores), n=4, eos=7), ref.select(logits, scores, 4, None, 7))


def test_the_first_step_and_the_last():
    """One live beam of four offers all; all finished: they stay, in order of their scores."""
    rng = np.random.default_rng(5)
    logits, scores = problem(rng, 3, 4, 700)
    first = np.full((3, 4), -np.inf, np.float32)
    first[:, 0] = 0
    check(cf.beam_select(dev(logits), dev(first)), ref.select(logits, first, 4))
    done = np.ones((3, 4), bool)
    check(cf.beam_select(dev(logits), dev(scores), done=dev(done), eos=5), ref.select(logits, scores, 4, done, 5))
    check(cf.beam_select(dev(logits), dev(scores), done=dev(done).view(torch.uint8), eos=5, n=9),
          ref.select(logits, scores, 9, done, 5))


def test_large_and_small_logits():
    rng = np.random.default_rng(6)
    for spread, shift in ((1e-3, 0), (30, 0), (3, 5e4), (3, -1e6), (1e30, 0), (1e-40, 0)):
        logits, scores = problem(rng, 2, 3, 1500, spread)
        logits = (logits + np.float32(shift)).astype(np.float32)
        note(f"beam magnitudes {spread} {shift}")
        want = ref.select(logits, scores, 3)
        if want[4] <= 2e-6:  # equal in FP64, or too near: of one beam only
            logits, scores = logits[:2], scores[:, :1]
            want = ref.select(logits, scores, 3)
        got = cf.beam_select(dev(logits), dev(scores), n=3)
        torch.cuda.synchronize()
        assert np.array_equal(got[0].cpu().numpy(), want[0]) and np.array_equal(got[1].cpu().numpy(), want[1])
        off = np.abs(got[2].cpu().numpy() - want[2])
        assert (off <= 3e-7 + np.abs(want[2]) * 2.0 ** -23).all()


@pytest.mark.parametrize("shape", [(), (1,), (3,), (300,), (7, 2, 5)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.uint8, torch.float16, torch.int64, torch.bool])
def test_reorder(shape, dtype):
    g = torch.Generator(device="cuda").manual_seed(1)
    states = torch.randint(0, 2 if dtype == torch.bool else 100, (9, *shape), generator=g, device="cuda").to(dtype)
    parents = torch.tensor([[3, 3, 0], [8, -1, 9], [1 << 30, 2, 7]], dtype=torch.int32, device="cuda")
    note(f"beam reorder {shape} {dtype}")
    got = cf.beam_reorder(states, parents)
    want = torch.zeros(9, *shape, dtype=dtype, device="cuda")
    for i, p in enumerate(parents.flatten().tolist()):
        if 0 <= p < 9:
            want[i] = states[p]
    assert torch.equal(got, want)
    if shape:  # a view of wider rows, and into one
        flat = torch.stack([states.flatten(1)] * 2, 1).flatten(1)
        half = flat[:, :states[0].numel()]
        out = torch.full_like(flat, 1)
        cf.beam_reorder(half, parents, out=out[:, :states[0].numel()])
        assert torch.equal(out[:, :states[0].numel()], want.flatten(1)) and bool((out[:, states[0].numel():] == 1).all())
    one = states[:1].expand(5, *shape)
    assert torch.equal(cf.beam_reorder(one, torch.tensor([4, 0], dtype=torch.int32, device="cuda")), states[:1].expand(2, *shape))


def test_refused_tensors():
    x, s = torch.zeros(4, 10, device="cuda"), torch.zeros(2, 2, device="cuda")
    for bad in (dict(scores=s[:1]), dict(scores=s.t()[:, :1]), dict(done=torch.zeros(2, 1, dtype=torch.bool, device="cuda")),
                dict(logits=x.t())):
        with pytest.raises((ValueError, TypeError)):
            cf.beam_select(**{**dict(logits=x, scores=s), **bad})
    for bad in (dict(scores=s.double()), dict(done=s), dict(logits=x.half()), dict(done=s.bool().cpu())):
        with pytest.raises(TypeError):
            cf.beam_select(**{**dict(logits=x, scores=s), **bad})
    for bad in (dict(n=0), dict(n=65)):
        with pytest.raises((cf.Cfp32Error, ValueError, RuntimeError)):
            cf.beam_select(x, s, **bad)
    i = torch.zeros(3, dtype=torch.int32, device="cuda")
    for bad in ((x.t(), i), (x, i, torch.zeros(2, 10, device="cuda")), (x, i, torch.zeros(3, 10, device="cuda").half())):
        with pytest.raises(ValueError):
            cf.beam_reorder(*bad)
    with pytest.raises(TypeError):
        cf.beam_reorder(x, i.long())
    with pytest.raises(cf.Cfp32Error):
        cf.beam_reorder(x, torch.zeros(4, dtype=torch.int32, device="cuda"), out=x)


def test_streams_workspaces_and_a_graph():
    rng = np.random.default_rng(7)
    logits, scores = problem(rng, 4, 4, 6000)
    x, s, d = dev(logits), dev(scores), torch.zeros(4, 4, dtype=torch.bool, device="cuda")
    hist = torch.arange(16 * 9, dtype=torch.int32, device="cuda").view(16, 9)

    def step(stream=None, ws=None):
        r = cf.beam_select(x, s, done=d, eos=3, workspace=ws, stream=stream)
        return (*r, cf.beam_reorder(hist, r[0], stream=stream))

    note("beam streams and graph")
    want = step()
    need = cf.cfp32_beam_select_workspace_bytes(4, 4, 6000, 4)
    ws = cf.Workspace()
    ws.get(need, x.device).fill_(0xFF)
    assert all(torch.equal(a, b) for a, b in zip(step(ws=ws), want))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = step(st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(g, stream=st):
            outs = step(st, ws)
    for i in range(4):
        x.normal_()
        d.copy_(torch.rand(4, 4, device="cuda") < 0.3)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, step()))
