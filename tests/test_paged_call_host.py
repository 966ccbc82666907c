"""The compiled way from tensors to the paged cache's C ABI (``native/paged_call.cpp``) on a host without a GPU:
built for host tensors over a stand-in for the library (``tests/paged_call_stub.cpp``), so that calls pass the
device check and reach the entry points, which no kernel follows."""
from __future__ import annotations

import ctypes
import importlib.util
import os
import subprocess
import sys
import sysconfig

import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC = os.path.join(ROOT, "geometric_map_reduce_amd", "native", "paged_call.cpp")
STUB = os.path.join(HERE, "paged_call_stub.cpp")


@pytest.fixture(scope="module")
def built(tmp_path_factory):
    """The folder with the module and its stand-in library."""
    from torch.utils.cpp_extension import include_paths
    to = tmp_path_factory.mktemp("paged_call")
    inc = ["-I", os.path.join(ROOT, "include"), "-isystem", sysconfig.get_paths()["include"]]
    for p in include_paths():
        inc += ["-isystem", p]
    common = ["g++", "-O1", "-shared", "-fPIC", "-std=c++17", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *inc]
    libs = ["-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    for cmd in ([*common, STUB, "-o", str(to / "libstub.so")],
                [*common, "-DPAGED_CALL_DEVICE=c10::DeviceType::CPU", SRC, "-o", str(to / "_paged_call.so"), *libs, "-L", str(to),
                 "-l:libstub.so", "-Wl,-rpath,$ORIGIN"]):
        res = subprocess.run(cmd, capture_output=True, text=True)
        assert res.returncode == 0, res.stderr
    return str(to)


def load(folder):
    spec = importlib.util.spec_from_file_location("_paged_call", os.path.join(folder, "_paged_call.so"))
    short = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(short)
    short.bind(lambda dev: 0)
    return short, ctypes.CDLL(os.path.join(folder, "libstub.so"))


def arguments(outputs=False):
    """Plain right arguments of the four calls, by name; their outputs given or not."""
    bf, i32 = torch.bfloat16, torch.int32
    k = torch.zeros((4, 16, 2, 64), dtype=bf)
    table, lens, starts = torch.zeros((1, 4), dtype=i32), torch.ones(1, dtype=i32), torch.tensor([0, 1], dtype=i32)
    w = torch.zeros((4, 2, 16))
    rows, q = torch.zeros((1, 2, 64), dtype=bf), torch.zeros((1, 4, 64), dtype=bf)
    p = torch.full((1, 2, 8), 0.125)
    o = [q.clone(), torch.zeros((1, 4)), torch.zeros((1, 2, 4), dtype=i32), lens.clone(), torch.zeros((1, 2), dtype=i32), lens.clone()]
    if not outputs:
        o = [None] * 6
    return dict(
        append=[rows, rows.clone(), k, k.clone(), None, table, lens, None, None, starts],
        attention=[q, k, k.clone(), None, table, lens, None, None, starts, 1, 16, None, 0, 0.0, *o[:2]],
        evict=[k, k.clone(), w, table, lens, None, None, table.clone(), 4, 0, 0, *o[2:4]],
        verify=[p, p[:, :1].contiguous(), torch.zeros((1, 1), dtype=i32), lens, torch.zeros((1, 1)), torch.zeros(1), *o[4:]])


def test_plain_calls_reach_the_library(built):
    short, stub = load(built)
    stub.stub_set(0)
    a = arguments()
    assert short.append(*a["append"]) is True
    out, lse = short.attention(*a["attention"])
    assert out.shape == (1, 4, 64) and out.dtype == torch.bfloat16 and lse.shape == (1, 4)
    kept, lens = short.evict(*a["evict"])
    assert kept.shape == (1, 2, 4) and lens.shape == (1,)
    tokens, accepted = short.verify(*a["verify"])
    assert tokens.shape == (1, 2) and accepted.shape == (1,)
    assert stub.stub_calls() == 4
    a = arguments(outputs=True)
    for name in ("attention", "evict", "verify"):
        got = getattr(short, name)(*a[name])
        assert got[0] is a[name][-2] and got[1] is a[name][-1]


def every_batched_argument(folder):
    """Each tensor of each call in turn is one that torch.vmap batches: it has no memory of its own.
    Every such call is handed back, and nothing reaches the library."""
    short, stub = load(folder)
    stub.stub_set(0)
    for name, args in arguments(outputs=True).items():
        for at, x in enumerate(args):
            if not isinstance(x, torch.Tensor):
                continue

            def call(t):
                assert type(t) is torch.Tensor
                got = getattr(short, name)(*args[:at], t, *args[at + 1:])
                assert got is None, (name, at, got)
                print(name, at, flush=True)
                return t
            torch.vmap(call)(torch.stack([x, x]))
    assert stub.stub_calls() == 0


def test_batched_tensors_are_handed_back(built):
    """In a process of its own: an exception without the interpreter's lock would end it."""
    code = f"import sys; sys.path.insert(0, {HERE!r}); import test_paged_call_host as t; t.every_batched_argument({built!r})"
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, f"ended with {res.returncode} after\n{res.stdout}\n{res.stderr[-2000:]}"


INVALID, UNSUPPORTED, ALLOC, HIP, SCRATCH = -1, -2, -3, -4, -5


@pytest.mark.parametrize("outputs", [False, True])
def test_statuses(built, outputs):
    """What an entry point refuses before it enqueues anything is handed back, to be named by the long way.  A HIP error
    may come after a launch: it is given back as it is, and the call is not repeated."""
    short, stub = load(built)
    for status in (INVALID, UNSUPPORTED, ALLOC, HIP, SCRATCH):
        for name, args in arguments(outputs).items():
            stub.stub_set(status)
            got = getattr(short, name)(*args)
            assert stub.stub_calls() == 1
            assert got is None if status != HIP else type(got) is int and got == HIP, (name, status, got)


@pytest.mark.parametrize("name,call", [
    ("append", lambda m, a: m.keops_cache_append(*a[:4], *a[5:7], a[9])),
    ("attention", lambda m, a: m.keops_paged_attention(*a[:3], *a[4:6], a[8], 1, 16)),
    ("evict", lambda m, a: m.keops_cache_evict(*a[:5], a[7], 4)),
    ("verify", lambda m, a: m.keops_verify_draft(*a[:6]))])
def test_a_hip_error_is_raised_once(built, monkeypatch, name, call):
    from geometric_map_reduce_amd import KeopsError, binding, paged
    short, stub = load(built)
    monkeypatch.setattr(paged, "_short", short)
    monkeypatch.setattr(binding, "status_string", lambda rc: "HIP error")
    monkeypatch.setattr(paged, "_run", lambda *a: pytest.fail("the call went the long way too"))
    stub.stub_set(HIP)
    with pytest.raises(KeopsError) as e:
        call(paged, arguments()[name])
    assert e.value.status == HIP and stub.stub_calls() == 1
