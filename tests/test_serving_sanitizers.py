"""The host side of the rotary, 8-bit cache and beam calls under AddressSanitizer
and UndefinedBehaviorSanitizer, on the CPU: argument checks (serving_api.hip) and
plans (attention8_plans.hip, beam_plans.hip), with launcher stubs that abort if
reached (tests/sanitize/serving_driver.cpp)."""
import os
import shutil

import pytest

from test_sanitizers import CSRC, LLVM, SAN, SAN_ENV, _clean, _run


def test_serving_host_code_under_sanitizers(tmp_path):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc) or not os.path.exists(os.path.join(LLVM, "clang")):
        pytest.skip("the ROCm compilers are not available")
    san_host = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer"]
    objs = []
    for src in ("api.hip", "plans.hip", "attention_api.hip", "attention_plans.hip", "cache_plans.hip", "serving_api.hip",
                "attention8_plans.hip", "beam_plans.hip"):
        objs.append(str(tmp_path / (src + ".o")))
        _run([hipcc, "--offload-arch=gfx950", "-std=c++17", "-O1", "-g", "-fPIC", "-ffp-contract=off", *san_host,
              "-c", os.path.join(CSRC, src), "-o", objs[-1]])
    for src in ("launcher_stubs.cpp", "attention_stubs.cpp", "serving_stubs.cpp", "serving_driver.cpp"):
        objs.append(str(tmp_path / (src + ".o")))
        _run([os.path.join(LLVM, "clang++"), "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined",
              "-fno-sanitize-recover=undefined", "-I/opt/rocm/include", "-D__HIP_PLATFORM_AMD__", "-c",
              os.path.join(SAN, src), "-o", objs[-1]])
    exe = str(tmp_path / "serving_driver")
    _run([os.path.join(LLVM, "clang++"), "-fsanitize=address,undefined", *objs, "-L/opt/rocm/lib",
          "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib", "-o", exe])
    import torch
    r = _run([exe] + ([] if torch.cuda.is_available() else ["no-device"]), env={**os.environ, **SAN_ENV})
    _clean(r.stderr)
    assert ", 0 failure(s)" in r.stderr
