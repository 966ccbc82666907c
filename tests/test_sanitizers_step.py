"""The host side of the C ABI around the paged cache (``step_api.cpp`` and ``paged_api.cpp`` in
``geometric_map_reduce_amd/csrc``) in an address- and undefined-behaviour-sanitizer build of their host code, driven on the
CPU with valid, odd and wild arguments (``tests/sanitize/step_host_driver.cpp``)."""
from __future__ import annotations

import os
import subprocess

import pytest

from test_sanitizers import CLANGXX, CSRC, HIPCC, OBJ, ROCM, ROOT, SAN, _run


def test_step_host_under_asan_ubsan(tmp_path):
    if os.path.exists("/dev/kfd"):
        pytest.skip("a GPU device node is present: this driver runs on hosts without a GPU only")
    if not (os.path.exists(CLANGXX) and os.path.exists(HIPCC)):
        pytest.skip("ROCm clang / hipcc not available")
    apis = ("paged_api.cpp", "step_api.cpp")
    objs = sorted(os.path.join(OBJ, f) for f in os.listdir(OBJ) if f.endswith(".o") and f[:-2] not in apis) if os.path.isdir(OBJ) else []
    if not objs:
        pytest.skip("library objects not built")
    inc = ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
    built = []
    for api in apis:
        built.append(str(tmp_path / (api + ".o")))
        # sanitizers on the host code only (each -fsanitize= after -Xarch_host)
        _run([HIPCC, "-x", "hip", "--offload-arch=gfx950", "-fPIC", "-O1", "-g", "-fno-omit-frame-pointer",
              "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-std=c++17", *inc,
              "-c", os.path.join(CSRC, api), "-o", built[-1]])
    drv, exe = str(tmp_path / "driver.o"), str(tmp_path / "step_host_driver")
    _run([CLANGXX, "-O1", "-g", "-fno-omit-frame-pointer", "-fPIC", "-fsanitize=address,undefined",
          "-D__HIP_PLATFORM_AMD__", "-std=c++17", "-I", os.path.join(ROCM, "include"), *inc,
          "-c", os.path.join(SAN, "step_host_driver.cpp"), "-o", drv])
    _run([CLANGXX, "-fsanitize=address,undefined", drv, *built, *objs, "-L", os.path.join(ROCM, "lib"),
          "-Wl,-rpath," + os.path.join(ROCM, "lib"), "-lamdhip64", "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    res = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
    if res.returncode == 77:
        pytest.skip(res.stdout.strip())
    assert res.returncode == 0, f"driver failed ({res.returncode}):\n{res.stdout}\n{res.stderr[-4000:]}"
    assert "ok" in res.stdout and "runtime error" not in res.stderr
