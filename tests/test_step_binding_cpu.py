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
