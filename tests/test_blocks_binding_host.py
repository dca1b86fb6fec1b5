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


@pytest.fixture
def allocation(monkeypatch):
    """Stand-ins for torch's allocation: its private function and torch.empty, and
    how many dispatch modes are on."""
    state = types.SimpleNamespace(modes=0, fast=[], plain=[])

    def fast(shape, strides, dtype):
        state.fast.append((shape, strides, dtype))
        return "fast"

    def empty(shape, dtype, device):
        state.plain.append((shape, dtype))
        return "plain"

    torch = types.SimpleNamespace(empty=empty, _C=types.SimpleNamespace(
        _cuda_getDevice=lambda: 0, _len_torch_dispatch_stack=lambda: state.modes))
    monkeypatch.setattr(r, "_torch", torch)
    monkeypatch.setattr(r, "_fast_empty", fast)
    return state


def test_allocation_under_a_dispatch_mode_is_seen_by_it(allocation):
    assert r._new((3, 4), "t", Tensor()) == "fast" and allocation.fast == [((3, 4), (4, 1), "t")]
    allocation.modes = 1
    assert r._new((3, 4), "t", Tensor()) == "plain" and allocation.plain == [((3, 4), "t")]


@pytest.mark.parametrize("error", [TypeError, RuntimeError])
def test_allocation_falls_back_where_the_private_function_takes_other_arguments(allocation, monkeypatch, error):
    tried = []

    def fast(*args):
        tried.append(args)
        raise error("other arguments")

    monkeypatch.setattr(r, "_fast_empty", fast)
    if error is RuntimeError:   # (memory that runs out is not hidden)
        with pytest.raises(RuntimeError):
            r._new((5,), "t", Tensor())
        assert r._fast_empty is fast
        return
    assert r._new((5,), "t", Tensor()) == "plain" and r._new((5, 2), "t", Tensor()) == "plain"
    assert len(tried) == 1 and allocation.plain == [((5,), "t"), ((5, 2), "t")]


def test_a_callers_mistake_does_not_turn_the_private_function_off(allocation, monkeypatch):
    def refuse(*args, **kwargs):
        raise TypeError("not a dtype")

    monkeypatch.setattr(r, "_fast_empty", refuse)
    monkeypatch.setattr(r._torch, "empty", refuse)
    with pytest.raises(TypeError, match="not a dtype"):
        r._new((5,), "no dtype", Tensor())
    assert r._fast_empty is refuse


def test_allocation_without_a_way_to_see_dispatch_modes(monkeypatch):
    """A torch that cannot be asked for dispatch modes is not passed by."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(r, "_torch", None)
    monkeypatch.setattr(r, "_fast_empty", None)
    monkeypatch.delattr(torch._C, "_len_torch_dispatch_stack")
    r._use_torch()
    assert r._torch is torch and r._fast_empty is None


def test_workspaces_that_are_less_than_they_seem_are_refused():
    """A workspace's size is its number of elements: an expanded tensor has fewer
    behind it, and a strided one has neighbours between them."""
    torch = pytest.importorskip("torch")
    x, w, d = (torch.zeros(s, dtype=torch.bfloat16) for s in ((4, 8), (6, 8), (8, 6)))
    p = torch.zeros(8, dtype=torch.bfloat16)
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(1 << 20, dtype=torch.uint8)[::2],
               torch.zeros((64, 64), dtype=torch.float32).T):
        for call in (lambda: r.rope3d_gated_ffn(x, w, w, d, workspace=ws),
                     lambda: r.rope3d_gated_ffn_backward(x, x, w, w, d, workspace=ws),
                     lambda: r.rope3d_block_norm_backward(x, dn=x, pre_weight=p, workspace=ws)):
            with pytest.raises(ValueError, match="workspace"):
                call()
