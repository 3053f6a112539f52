"""CPU checks of calls around the attention and the experts that came up in use:
what they refuse, and what the binding passes on."""
import ctypes

import moe_decode_amd as md

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
