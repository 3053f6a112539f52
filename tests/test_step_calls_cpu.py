"""CPU checks of calls around the attention and the experts that came up in use:
what they refuse, and what the binding passes on."""
import ctypes

import torch

import moe_decode_amd as md

from . import test_streams_cpu as streams
from .test_attn_abi_cpu import FAKE, ODD, _b, _st

OUT = FAKE + (1 << 24)


def test_tree_window_refusals():
    L = md.lib()

    def tree(par=FAKE, window=4, sinks=2, masks=OUT, words=1, pos=OUT, **kw):
        return _st(L.md_kv_tree_window(ctypes.byref(_b(**kw)), par, window, sinks, masks, words, pos, None))
    assert _st(L.md_kv_tree_window(None, FAKE, 4, 2, OUT, 1, OUT, None)) == "MD_ERR_INVALID_ARG"
    for kw, want in [(dict(window=-1), "INVALID_ARG"), (dict(sinks=-1), "INVALID_ARG"), (dict(S=0), "SHAPE"),
                     (dict(max_q=1025, words=17), "UNSUPPORTED"), (dict(max_q=65), "SHAPE"), (dict(words=0), "SHAPE"),
                     (dict(par=None), "INVALID_ARG"), (dict(masks=None), "INVALID_ARG"), (dict(masks=ODD), "ALIGNMENT"),
                     (dict(par=FAKE + 2), "ALIGNMENT"), (dict(pos=OUT + 1), "ALIGNMENT")]:
        assert tree(**kw) == "MD_ERR_" + want, kw
    assert tree(rows=0, par=None, masks=None) == "MD_OK"
    assert tree(rows=0, window=-1, par=None, masks=None) == "MD_ERR_INVALID_ARG"


def test_workspace_sizes_of_masked_and_routed_calls():
    """What a caller that brings its own workspace asks for: the C functions' sizes."""
    L, sz = md.lib(), ctypes.c_size_t(0)
    c = streams._cache()
    b = md.KVBatch(streams._i32([0, 3]), streams._i32([3]), torch.zeros(1, 4000, dtype=torch.int32), 3, 100000)
    tree = torch.zeros(3, 2, dtype=torch.int64)
    for kw, mask in [(dict(window=50000, sinks=70), (50000, 70, 0, None)), (dict(tree=tree), (0, 0, 2, tree.data_ptr())),
                     (dict(window=3, sinks=1 << 40), (3, (1 << 31) - 1, 0, None))]:
        m = md.KVMaskDesc(*mask)
        assert L.md_kv_attention_masked_workspace_size(c._ref, b.desc(3), 4, ctypes.byref(m), 0, ctypes.byref(sz)) == 0
        assert md.kv_attention_workspace_size(c, b, 3, 4, **kw) == sz.value, kw
    many = md.KVBatch(streams._i32([0, 200]), streams._i32([3]), torch.zeros(1, 4000, dtype=torch.int32), 200, 100000)
    tree = torch.zeros(200, 4, dtype=torch.int64)
    assert md.kv_attention_workspace_size(c, many, 200, 4, tree=tree) > md.kv_attention_workspace_size(c, many, 200, 4) > 0
    layer = streams._moe()
    assert L.md_moe_routed_workspace_size(ctypes.byref(layer.desc()), 5, ctypes.byref(sz)) == 0
    assert md.moe_workspace_size(layer, 5, routed=True) == sz.value > 0
