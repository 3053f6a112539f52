"""What the binding refuses or passes on around the attention and the experts,
checked without a GPU on a library that only takes notes."""
import pytest
import torch

import moe_decode_amd as md

from . import test_streams_cpu as streams
from .test_streams_cpu import _notes  # noqa: F401  (an autouse fixture)

Q = torch.zeros(3, 4, 64)


def test_masks_of_no_words_are_no_missing_tree():
    """An empty tensor's address is null: the call would have been a causal one."""
    with pytest.raises(ValueError, match="words"):
        md.kv_attention(streams._cache(), streams._batch(), Q, tree=torch.zeros(3, 0, dtype=torch.int64))
    assert not streams.NOTES.streams


@pytest.mark.parametrize("tree", [None, torch.zeros(3, 1, dtype=torch.int64)])
@pytest.mark.parametrize("window,sinks", [((1 << 32) + 5, 0), ((1 << 32) + 5, (1 << 33) + 2), (7, 1 << 32), (1 << 31, 4)])
def test_windows_and_sinks_past_32_bits_reach_every_position(tree, window, sinks, monkeypatch):
    """ctypes would pass their low 32 bits, a window of 5 for one of 2^32 + 5."""
    got, most = [], (1 << 31) - 1

    class Library(streams._Library):
        def __getattr__(self, name):
            call = super().__getattr__(name)

            def noted(*args):
                if name == "md_kv_attention":
                    got.append((args[8], 0))
                elif name == "md_kv_attention_workspace_size":
                    assert args[4] == min(window, most)
                elif name == "md_kv_attention_masked":
                    got.append((args[7]._obj.window, args[7]._obj.sinks))
                elif name == "md_kv_tree_window":
                    got.append(args[2:4])
                return call(*args)
            return noted
    monkeypatch.setattr(md, "lib", lambda: Library())
    md.kv_attention_workspace_size(streams._cache(), streams._batch(), 3, 4, window=window)
    md.kv_attention(streams._cache(), streams._batch(), Q, window=window, sinks=sinks, tree=tree)
    md.kv_tree(streams._batch(), streams._i32([-1, 0, 0]), window=window, sinks=sinks)
    assert got == [(min(window, most), min(sinks, most))] * 2
