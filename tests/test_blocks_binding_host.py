"""The block operators' binding on stand-ins for torch's CUDA tensors and streams (no GPU)."""
from __future__ import annotations

import contextlib
import types

import pytest

import rope_rope3d_apply_gb300 as r


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class ExternalStream(Stream):
    def __init__(self, handle, device=None):
        super().__init__(handle)


class Tensor:
    def __init__(self, is_cuda=True):
        self.is_cuda, self.device, self.used_on = is_cuda, types.SimpleNamespace(index=0), []

    def record_stream(self, stream):
        assert self.is_cuda
        self.used_on.append(stream.cuda_stream)


HERE = 1


@pytest.fixture
def stand_in(monkeypatch):
    """torch as far as _elsewhere uses it; stream 1 is the current one."""
    entered = []

    @contextlib.contextmanager
    def current(stream):
        entered.append(stream.cuda_stream)
        yield

    torch = types.SimpleNamespace(
        Tensor=Tensor, _C=types.SimpleNamespace(_cuda_getCurrentRawStream=lambda i: HERE),
        cuda=types.SimpleNamespace(Stream=Stream, ExternalStream=ExternalStream, stream=current,
                                   current_stream=lambda device: Stream(HERE)))
    monkeypatch.setattr(r, "_torch", torch)
    return entered


def test_inputs_of_a_call_on_another_stream_are_marked_as_used_there(stand_in):
    """A temporary passed with stream= may be freed as soon as the call returns, while
    the other stream still reads it: it is marked before anything is launched. Streams
    of torch's own live as long as the process; one that torch did not make may be gone
    when the memory is freed, and is left to the caller."""
    x, y, w, out = Tensor(), Tensor(), Tensor(), Tensor()
    host = Tensor(is_cuda=False)
    seen = {}

    def call(**args):
        seen.update(args)
        assert all(t.used_on == ([2] if marked else []) for t in (x, y, w))
        return out, None

    marked = True
    assert r._elsewhere(call, dict(x=x, y=y, post_weight=w, gate=None, scale=host, eps=1e-6, stream=Stream(2))) == (out, None)
    assert stand_in == [2] and set(seen) == {"x", "y", "post_weight", "gate", "scale", "eps"}
    assert out.used_on == [HERE] and host.used_on == []
    for t in (x, y, w, out):
        t.used_on.clear()
    marked = False
    for stream in (3, ExternalStream(3)):
        assert r._elsewhere(call, dict(x=x, y=y, post_weight=w, gate=None, scale=host, eps=1e-6, stream=stream)) == (out, None)
    assert stand_in == [2, 3, 3] and out.used_on == [HERE, HERE]
    # the current stream needs none of it
    assert r._elsewhere(call, dict(x=x, stream=Stream(HERE))) is None
