"""Where a call on a stream that it is given makes its outputs, on a host without a GPU: memory of the current
stream's pool may still be in use by work that is queued there, of which the other stream knows nothing."""
from __future__ import annotations

import contextlib

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from geometric_map_reduce_amd import paged


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def calls(monkeypatch):
    """The four calls on host tensors, with everything below the allocations left out; what they make, and on which
    stream."""
    current, made, kept = [Stream(1)], [], []

    @contextlib.contextmanager
    def stream(s):
        current.append(s or current[-1])
        yield
        current.pop()

    class Watch(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            out = func(*args, **(kwargs or {}))
            if "empty" in func.name():
                made.append((tuple(out.shape), current[-1].cuda_stream))
            return out

    def graph_workspace(name, dev, *args):
        made.append((name, current[-1].cuda_stream))
        return None, 0, torch.empty(1)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: current[-1])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: kept.append((tuple(t.shape), s.cuda_stream)))
    monkeypatch.setattr(paged, "_cache", lambda *a, **k: (b"", 0, 3, (2, 64, torch.bfloat16), 16, 4))
    monkeypatch.setattr(paged, "_rows", lambda *a: (16, 64))
    monkeypatch.setattr(paged, "_vec", lambda *a: 16)
    monkeypatch.setattr(paged, "_table", lambda *a: (16, 4, 4))
    monkeypatch.setattr(paged, "_graph_workspace", graph_workspace)
    monkeypatch.setattr(paged, "_run", lambda *a: None)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    k, i = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16), torch.zeros((3, 4), dtype=torch.int32)
    q, w, p = torch.zeros((5, 4, 64), dtype=torch.bfloat16), torch.zeros((4, 2, 16)), torch.zeros((3, 3, 8))

    def run(s):
        with Watch():
            paged.keops_paged_attention(q, k, k, i, i, i, 2, 8, stream=s)
            paged.keops_paged_attention(q.transpose(0, 1).contiguous().transpose(0, 1), k, k, i, i, i, 2, 8, stream=s)
            paged.keops_cache_evict(k, k, w, i, i, i, 4, stream=s)
            paged.keops_verify_draft(p, None, i[:, :2], i, i, i, stream=s)
        return made, kept
    return run


def test_outputs_are_made_on_the_stream_of_the_call(calls):
    made, kept = calls(Stream(2))
    shapes = [(5, 4, 64), (5, 4), (5, 4, 64), (5, 4), (3, 2, 4), (3,), (3, 3), (3,)]
    assert [m[0] for m in made if isinstance(m[0], tuple) and m[0] != (1,)] == shapes
    assert all(s == 2 for _, s in made), made
    # and belong to the caller's stream too, which reads them
    assert kept == [(s, 1) for s in shapes]


def test_the_current_stream_needs_nothing(calls, monkeypatch):
    monkeypatch.setattr(paged, "_native", lambda: None)
    monkeypatch.setattr(paged, "_short", None)
    for s in (None, Stream(1)):
        made, kept = calls(s)
        assert all(s == 1 for _, s in made) and not kept


@pytest.mark.parametrize("current", [0, 1])
def test_the_default_streams_handle_is_the_default_stream(calls, monkeypatch, current):
    """0 is a handle, but torch.cuda.ExternalStream takes it for none and hands out a stream of its pool."""
    now = [Stream(current)]

    @contextlib.contextmanager
    def stream(s):
        now.append(s or now[-1])
        yield
        now.pop()
    empty = torch.Tensor.new_empty
    seen = []

    def new_empty(t, *a, **k):
        seen.append(now[-1].cuda_stream)
        return empty(t, *a, **k)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: now[-1])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda dev=None: Stream(0))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(handle or 999))
    monkeypatch.setattr(torch.Tensor, "new_empty", new_empty)
    calls(0)
    assert seen and all(s == 0 for s in seen), seen
    seen.clear()
    calls(7)
    assert seen and all(s == 7 for s in seen), seen
