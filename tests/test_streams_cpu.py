"""Calls with `stream=`: what the binding allocates for a call has to belong to
the stream that its kernels run on, or the allocator hands a released workspace
to the next tensor of the current stream while they still use it.  Checked here
without a GPU, on a library and an allocator that only take notes."""
import contextlib
import ctypes
import types

import numpy as np
import pytest
import torch

import moe_decode_amd as md


class _Tensor(torch.Tensor):
    def record_stream(self, stream):
        NOTES.recorded.append((self.data_ptr(), stream))


NOTES = types.SimpleNamespace()
SIDE, NOW = types.SimpleNamespace(cuda_stream=123), types.SimpleNamespace(cuda_stream=7)


class _Library:
    """Every entry point succeeds and notes the stream it got; workspaces are
    4096 bytes."""

    def __getattr__(self, name):
        def call(*args):
            if name == "md_row_bytes":
                return args[1]
            if name.endswith("workspace_size"):
                args[-1]._obj.value = 4096
            else:
                NOTES.streams.append(123 in args)
            return 0
        return call


@pytest.fixture(autouse=True)
def _notes(monkeypatch):
    NOTES.current, NOTES.made, NOTES.recorded, NOTES.streams = [], [], [], []
    empty = torch.empty

    @contextlib.contextmanager
    def on(stream):
        NOTES.current.append(stream)
        yield
        NOTES.current.pop()

    def noting(make):
        def made(*args, **kw):
            t = make(*args, **kw).as_subclass(_Tensor)
            NOTES.made.append((t, NOTES.current[-1] if NOTES.current else None))
            return t
        return made
    monkeypatch.setattr(torch, "empty", noting(empty))
    monkeypatch.setattr(torch, "empty_like", noting(torch.empty_like))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: NOW)
    monkeypatch.setattr(md, "lib", lambda: _Library())
    monkeypatch.setattr(md, "_on", lambda device, stream: contextlib.nullcontext(
        (NOW if stream is None else stream).cuda_stream))


def _mat(rows, cols, count=1, type_="i8_row"):
    return md.DevQMatrix(type_, rows, cols, torch.zeros(rows * cols * count, dtype=torch.int8),
                         torch.zeros(rows * count), count)


def _ffn():
    return md.FFN("silu", _mat(256, 256), _mat(256, 256), _mat(256, 256))


def _moe():
    return md.MoELayer(256, 256, 4, 2, "silu", _mat(256, 256, 4), _mat(256, 256, 4), _mat(256, 256, 4),
                       torch.zeros(4, 256))


def _cache():
    return md.KVCache(torch.zeros(2, 2, 64, 64, dtype=torch.int8), torch.zeros(2, 2, 64, 64, dtype=torch.int8),
                      torch.zeros(2, 2), torch.zeros(2, 2))


def _i32(v):
    return torch.from_numpy(np.asarray(v, np.int32))


def _batch():
    return md.KVBatch(_i32([0, 3]), _i32([3]), _i32([[0, 1]]), 3, 128)


class _Event:
    cuda_event = 1


def _tier():
    t = md.ExpertTier.__new__(md.ExpertTier)
    t.host = t.slots = _moe()
    t.cache, t.copy_stream, t.copy_done = types.SimpleNamespace(state=ctypes.c_int(0)), None, None
    return t


X = torch.zeros(3, 256)
IDX, GATES = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
CALLS = {   # what is returned to the caller and what is let go: tensors of each
    "qgemv": (lambda **k: md.qgemv(_mat(256, 256), X, **k), 1, 1),
    "moe_route_topk": (lambda **k: md.moe_route_topk(X, torch.zeros(4, 256), None, 2, **k), 2, 1),
    "ffn_forward": (lambda **k: md.ffn_forward(_ffn(), X, **k), 1, 1),
    "moe_layer_forward": (lambda **k: md.moe_layer_forward(_moe(), X, **k), 1, 1),
    "moe_layer_forward residual": (lambda **k: md.moe_layer_forward(_moe(), X, residual=X, **k), 1, 1),
    "moe_layer_forward_timed": (lambda **k: md.moe_layer_forward_timed(_moe(), X, "router", _Event, _Event, **k), 1, 1),
    "add": (lambda **k: md.add(X, X, **k), 1, 0),
    "moe_experts_forward": (lambda **k: md.moe_experts_forward(_moe(), X, IDX, GATES, **k), 1, 1),
    "ExpertTier.forward": (lambda **k: _tier().forward(X, **k), 1, 1),
    "i8_quantize": (lambda **k: md.i8_quantize(X, **k), 2, 0),
    "i8_matmul": (lambda **k: md.i8_matmul(_mat(256, 256), torch.zeros(3, 256, dtype=torch.int8), torch.zeros(3), **k),
                  1, 0),
    "i8_linear": (lambda **k: md.i8_linear(_mat(256, 256), X, **k), 1, 1),
    "kv_attention": (lambda **k: md.kv_attention(_cache(), _batch(), torch.zeros(3, 4, 64), **k), 1, 1),
    "kv_read_pages": (lambda **k: md.kv_read_pages(_cache(), _i32([0, 1]), **k), 2, 0),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_tensors_of_a_call_belong_to_its_stream(name):
    call, kept, gone = CALLS[name]
    out = call(stream=SIDE)
    out = out if isinstance(out, tuple) else (out,)
    assert NOTES.streams == [True]
    assert len(NOTES.made) == kept + gone
    assert all(st is SIDE for _, st in NOTES.made), [(tuple(t.shape), st) for t, st in NOTES.made]
    # what goes to the caller is noted as in use on the stream it was current on, what is released is not
    assert sorted(NOTES.recorded) == sorted((t.data_ptr(), NOW) for t in out)


@pytest.mark.parametrize("name", list(CALLS))
def test_without_a_stream_nothing_is_switched(name):
    call, kept, gone = CALLS[name]
    call()
    assert NOTES.streams == [False] and len(NOTES.made) == kept + gone
    assert all(st is None for _, st in NOTES.made) and not NOTES.recorded
