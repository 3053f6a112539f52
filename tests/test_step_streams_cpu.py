"""Calls with `stream=` around the attention and the experts: what the binding
allocates for a call belongs to the stream that its kernels run on (checked
without a GPU, on the library and the allocator of test_streams_cpu.py that only
take notes)."""
import pytest
import torch

import moe_decode_amd as md

from . import test_streams_cpu as streams
from .test_streams_cpu import _notes  # noqa: F401  (an autouse fixture)

TREE = torch.zeros(3, 1, dtype=torch.int64)
CALLS = {   # what is returned to the caller and what is let go: tensors of each
    "qk_norm_rope": (lambda **k: md.qk_norm_rope(torch.zeros(3, 4, 64), torch.zeros(3, 2, 64), streams._i32([0, 1, 2]),
                                                 torch.zeros(32), **k), 2, 0),
    "moe_route": (lambda **k: md.moe_route(streams.X, torch.zeros(4, 256), md.Routing(2), **k), 2, 1),
    "moe_layer_forward": (lambda **k: md.moe_layer_forward(streams._moe(), streams.X, routing=md.Routing(2), **k), 1, 1),
    "token_logprobs": (lambda **k: tuple(md.token_logprobs(torch.zeros(3, 256), streams._i32([[1], [2], [3]]), top=2, **k)),
                       4, 1),
    "kv_attention tree": (lambda **k: md.kv_attention(streams._cache(), streams._batch(), torch.zeros(3, 4, 64), tree=TREE,
                                                      **k), 1, 1),
    "kv_attention sinks": (lambda **k: md.kv_attention(streams._cache(), streams._batch(), torch.zeros(3, 4, 64), window=4,
                                                       sinks=2, **k), 1, 1),
    "kv_tree": (lambda **k: md.kv_tree(streams._batch(), streams._i32([-1, 0, 0]), **k), 2, 0),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_tensors_of_a_call_belong_to_its_stream(name):
    call, kept, gone = CALLS[name]
    out = call(stream=streams.SIDE)
    out = out if isinstance(out, tuple) else (out,)
    notes = streams.NOTES
    assert notes.streams == [True] and len(notes.made) == kept + gone
    assert all(st is streams.SIDE for _, st in notes.made)
    assert sorted(notes.recorded) == sorted((t.data_ptr(), streams.NOW) for t in out)
    notes.made, notes.recorded, notes.streams = [], [], []
    call()
    assert notes.streams == [False] and len(notes.made) == kept + gone
    assert all(st is None for _, st in notes.made) and not notes.recorded
