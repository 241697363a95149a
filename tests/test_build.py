"""The build, on the host with the compilers replaced: the C library stands
without what only the native tensor helpers need, and what is recorded beside
it is its own."""
import importlib.util
import json
import os
import subprocess

import pytest
import torch

import compensated_fp32_projection_amd as cf
from compensated_fp32_projection_amd import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """An old library, helpers and record, and compilers that write what they are asked for."""
    for name, attr in (("libcfp32.so", "LIB"), ("_helpers.so", "HELPERS"), ("build_info.json", "BUILD_INFO")):
        monkeypatch.setattr(build, attr, str(tmp_path / name))
        (tmp_path / name).write_text("old")
    ran = []

    def run(cmd, **kw):
        if "-o" not in cmd:
            return subprocess.CompletedProcess(cmd, 0, "", "")
        ran.append(os.path.basename(cmd[0]))
        fails = ran[-1] in run.fails
        if not fails:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write("new " + ran[-1])
        return subprocess.CompletedProcess(cmd, int(fails), "", "it fails" if fails else "")

    run.fails, run.ran = (), ran
    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "hipcc", lambda: "/nowhere/hipcc")
    return run


def recorded():
    with open(build.BUILD_INFO) as f:
        return json.load(f)["library_sha256"]


def test_everything_is_built_and_recorded(tree):
    build.build()
    assert tree.ran == ["hipcc", "g++"] and recorded() == build.file_hash(build.LIB)
    assert open(build.LIB).read() == "new hipcc" and open(build.HELPERS).read() == "new g++"


def test_helpers_that_do_not_compile_leave_the_library_and_its_record(tree):
    tree.fails = ("g++",)
    with pytest.raises(RuntimeError):
        build.build()
    assert open(build.LIB).read() == "new hipcc" and recorded() == build.file_hash(build.LIB)
    assert not os.path.exists(build.HELPERS)  # the old ones are bound to the old library's calls


def test_a_library_that_does_not_compile_leaves_all_as_it_was(tree):
    tree.fails = ("hipcc",)
    with pytest.raises(RuntimeError):
        build.build()
    assert all(open(p).read() == "old" for p in (build.LIB, build.HELPERS, build.BUILD_INFO))


@pytest.mark.parametrize("what", ["torch", "compiler", "headers"])
def test_the_library_needs_no_torch_headers_or_host_compiler(tree, monkeypatch, what, capsys):
    if what == "torch":
        find = importlib.util.find_spec
        monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    elif what == "compiler":
        monkeypatch.setattr(build.shutil, "which", lambda name: None)
    else:
        monkeypatch.setattr("sysconfig.get_paths", lambda: {"include": "/nowhere"})
    assert build.build() == build.LIB
    assert tree.ran == ["hipcc"] and recorded() == build.file_hash(build.LIB) and not os.path.exists(build.HELPERS)
    assert "native" in capsys.readouterr().err


def test_helpers_without_their_native_form(tmp_path, monkeypatch):
    """The Python form does the calls, after one warning."""
    monkeypatch.setattr(cf, "_HERE", str(tmp_path))
    monkeypatch.setattr(cf, "_helpers", None)
    x, i = torch.zeros(4, 2, 64), torch.zeros(3, dtype=torch.int32)
    with pytest.warns(RuntimeWarning, match="native"), pytest.raises(TypeError):
        cf.attention_prompt(x, x, x, i)
    n = cf._native()
    assert n.attention_prompt(x, x, x, i, None, True, None, None) is None
    for call in (n.attention_decode, n.cache_reserve, n.cache_append, n.cache_fork, n.cache_free, n.cache_compact):
        assert call(i) is None
