"""What a call on a given stream allocates for itself is taken under that stream, so that the
caching allocator neither hands it a block that the current stream has yet to finish with nor
gives its workspace away while its kernels run (no GPU: the streams, tensors and the library's
entries are stand-ins that record what happens to them)."""
from __future__ import annotations

import contextlib
from types import SimpleNamespace

import pytest
import torch

import fp8_weight_only_gemm_gb300 as w8
from fp8_weight_only_gemm_gb300 import binding

CURRENT, OTHER = 0x11, 0x22
DEVICE = torch.device("cuda", 0)


class Made:
    def __init__(self, size, stream):
        self.size, self.stream, self.recorded = size, stream, []

    def record_stream(self, s):
        self.recorded.append(s.cuda_stream)


def given(*shape):
    return SimpleNamespace(shape=torch.Size(shape), dtype=torch.bfloat16, device=DEVICE)


@pytest.fixture
def world(monkeypatch):
    """`made`: every tensor allocated; `calls`: (entry, stream handle)."""
    w = SimpleNamespace(active=[CURRENT], made=[], calls=[])

    @contextlib.contextmanager
    def under(s):
        w.active.append(s.cuda_stream)
        yield
        w.active.pop()

    def make(shape, dtype=None, device=None):
        w.made.append(Made(shape, w.active[-1]))
        return w.made[-1]

    def entry(name):
        def call(*a):
            w.calls.append((name, CURRENT if a[-1] is None else a[-1]))
            return 0
        return call

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: SimpleNamespace(cuda_stream=w.active[-1]))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: SimpleNamespace(cuda_stream=handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch, "empty", make)
    monkeypatch.setattr(binding, "kv_attention_workspace_bytes", lambda *a: 4096)
    monkeypatch.setattr(binding, "_marshal", SimpleNamespace(**{n: entry(n) for n in ("kv_append", "kv_attention", "gemm_w4")}))
    return w


CACHE = SimpleNamespace(_address=1, _index=0, head_dim=128)
CALLS = {
    "kv_attention": lambda s: w8.kv_attention(CACHE, given(6, 8, 128), given(3, 4), given(3), stream=s),
    "kv_append": lambda s: w8.kv_append(CACHE, given(6, 2, 128), given(6, 2, 128), given(3, 4), given(3), q=given(6, 8, 128), stream=s),
    "gemm_w4": lambda s: w8.gemm_w4(given(2, 256), given(96, 128), given(96, 2), stream=s),
}


@pytest.mark.parametrize("stream", [OTHER, SimpleNamespace(cuda_stream=OTHER), 0], ids=["handle", "stream", "default"])
@pytest.mark.parametrize("name", CALLS)
def test_allocated_under_the_calls_stream(world, name, stream):
    handle = getattr(stream, "cuda_stream", stream)
    out = CALLS[name](stream)
    assert world.calls == [(name, handle)]
    assert len(world.made) == (2 if name == "kv_attention" else 1)
    assert [t.stream for t in world.made] == [handle] * len(world.made)
    # what is returned may be in use on the current stream when it is dropped
    assert out in world.made and out.recorded == [CURRENT]


@pytest.mark.parametrize("stream", [None, CURRENT, SimpleNamespace(cuda_stream=CURRENT)], ids=["none", "handle", "stream"])
@pytest.mark.parametrize("name", CALLS)
def test_the_current_stream_needs_nothing_more(world, name, stream):
    CALLS[name](stream)
    assert world.calls == [(name, CURRENT)]
    assert all(t.stream == CURRENT and not t.recorded for t in world.made)
