"""The helpers' workspace, on the host with the allocator or the library
replaced: whose memory a buffer is, and calls of several threads."""
import contextlib
import gc
import shutil
import subprocess
import threading
import weakref

import pytest
import torch

import compensated_fp32_projection_amd as cf


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Buffer:
    """What torch.empty gives here: remembers the stream it was allocated under."""

    def __init__(self, nbytes, device, under):
        self.nbytes, self.device, self.under, self.used_on = nbytes, device, under, []

    def numel(self):
        return self.nbytes

    def data_ptr(self):
        return id(self)

    def record_stream(self, stream):
        self.used_on.append(stream)


@pytest.fixture
def allocator(monkeypatch):
    """Streams of the fake allocator: the current one, and what was allocated."""
    state = {"current": Stream(1), "made": []}

    @contextlib.contextmanager
    def under(stream):
        before, state["current"] = state["current"], stream or state["current"]
        yield
        state["current"] = before

    def empty(nbytes, dtype=None, device=None):
        state["made"].append(Buffer(nbytes, device, state["current"]))
        return state["made"][-1]

    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: state["current"])
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(cf, "_default_ws", {})
    return state


def test_a_buffer_is_memory_of_the_stream_it_is_for(allocator):
    """Its first kernel runs on that stream: memory of another may still be in use there."""
    side, dev = Stream(2), torch.device("cuda", 0)
    ws = cf.Workspace()
    assert ws.get(100, dev, side).under is side and ws.buf.used_on == [side]
    assert ws.get(300, dev, side).under is side and ws.get(10, dev, side) is ws.buf
    assert [b.nbytes for b in allocator["made"]] == [100, 300]
    assert cf.Workspace().get(5, dev).under is allocator["current"]


def test_the_attention_helpers_take_it_there(allocator):
    side, dev = Stream(2), torch.device("cuda", 0)
    cf._scratch(64, dev, None, side)
    cf._scratch(64, dev, cf.Workspace(), side)
    cf._scratch(64, dev, None, None)
    assert [b.under.cuda_stream for b in allocator["made"]] == [2, 2, 1]


STUB = """
#include <stdlib.h>
#include <string.h>
#include <unistd.h>
static volatile int inside, met;
int calls_met(void) { return met; }
static long call(void)
{
    if (__atomic_add_fetch(&inside, 1, __ATOMIC_SEQ_CST) > 1) met = 1;
    usleep(2000);
    __atomic_sub_fetch(&inside, 1, __ATOMIC_SEQ_CST);
    return 0;
}
"""
# The calls that launch several kernels over one workspace.
WITH_WORKSPACE = ["cfp32_linear", "cfp32_linear_ex", "cfp32_linear_geglu", "cfp32_attention_prompt", "cfp32_attention_decode",
                  "cfp32_cache_fork", "cfp32_cache_compact"]


@pytest.mark.skipif(not shutil.which("gcc"), reason="needs a C compiler")
def test_calls_that_use_a_workspace_do_not_run_at_once(tmp_path, monkeypatch):
    """Two threads on one stream share its workspace: what a call launches over
    it must not be mixed with another's.  (A library in the place of the real
    one, whose calls notice each other.)"""
    src, lib = tmp_path / "stub.c", str(tmp_path / "stub.so")
    src.write_text(STUB + "".join(f"long {n}(void) {{ return call(); }}\n" for n in cf.EXPORTS))
    subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", lib], check=True)
    monkeypatch.setattr(cf, "LIB_PATH", lib)
    monkeypatch.setattr(cf, "_lib", None)
    cf.load_library()

    def work():
        for name in WITH_WORKSPACE * 5:
            f = getattr(cf, name)
            f(*[0] * f.__code__.co_argcount)

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert cf._lib.calls_met() == 0


def test_a_buffer_stays_while_a_call_is_made_with_it(allocator):
    """Also where another thread's call makes the workspace grow meanwhile."""
    dev, ws = torch.device("cuda", 0), cf.Workspace()
    for space in (ws, None):
        lent = cf._scratch(64, dev, space, None)
        first = weakref.ref((space or cf._default_workspace(dev, allocator["current"])).buf)
        allocator["made"].clear()
        (space or cf._default_workspace(dev, allocator["current"])).get(1000, dev, None)
        gc.collect()
        assert first() is not None and lent
        del lent


def test_the_native_form_gets_the_buffer_itself(allocator):
    """And declines (None) what has to be allocated first: the Python form does that."""
    dev = torch.device("cuda", 0)
    assert cf._scratch_buffer(64, 0, 1) is None
    cf._scratch(64, dev, None, None)
    assert cf._scratch_buffer(64, 0, 1) is cf._default_ws[(0, 1)].buf
    assert cf._scratch_buffer(65, 0, 1) is None and cf._scratch_buffer(64, 0, 2) is None
