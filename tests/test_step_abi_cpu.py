"""CPU checks of the entry points around the attention and the experts: every bad
argument is rejected with the documented status before anything is enqueued (no
call here reaches the GPU), and the binding's own checks."""
import ctypes

import pytest
import torch

import moe_decode_amd as md

from . import test_streams_cpu as streams
from .test_attn_abi_cpu import BAD_BATCH, BAD_CACHE, FAKE, ODD, _b, _c, _st

OUT = FAKE + (1 << 24)


def _rope(**kw):
    d = dict(head_dim=128, rot=128, interleaved=0, inv_freq=FAKE, factor=1.0, eps=1e-6, q_weight=FAKE, k_weight=FAKE)
    d.update(kw)
    return ctypes.byref(md.RopeDesc(*[d[n] for n, _ in md.RopeDesc._fields_]))


def _turn(r=None, pos=FAKE, rows=3, q=FAKE, hq=4, qs=512, k=FAKE, hk=2, ks=256, xt=0, qo=OUT, qos=512, ko=OUT + 65536,
          kos=256, yt=0, **kw):
    r = _rope(**kw) if r is None else r
    return _st(md.lib().md_qk_norm_rope(r, pos, rows, q, hq, qs, k, hk, ks, xt, qo, qos, ko, kos, yt, None))


def test_rope_refusals():
    L = md.lib()
    assert _st(L.md_qk_norm_rope(None, FAKE, 3, FAKE, 4, 512, FAKE, 2, 256, 0, OUT, 512, OUT, 256, 0, None)) == \
        "MD_ERR_INVALID_ARG"
    for kw, want in [(dict(xt=2), "INVALID_ARG"), (dict(yt=-1), "INVALID_ARG"), (dict(interleaved=2), "INVALID_ARG"),
                     (dict(factor=float("nan")), "INVALID_ARG"), (dict(eps=float("inf")), "INVALID_ARG"),
                     (dict(eps=-1.0), "INVALID_ARG"), (dict(rows=-1), "SHAPE"), (dict(hq=0), "SHAPE"),
                     (dict(hk=-1), "SHAPE"), (dict(head_dim=0), "SHAPE"), (dict(rot=136), "SHAPE"), (dict(rot=-8), "SHAPE"),
                     (dict(rows=(1 << 20) + 1), "UNSUPPORTED"), (dict(hq=1025), "UNSUPPORTED"),
                     (dict(hk=1025), "UNSUPPORTED"), (dict(head_dim=264, rot=8), "UNSUPPORTED"),
                     (dict(head_dim=100, rot=8), "UNSUPPORTED"), (dict(rot=12), "UNSUPPORTED"), (dict(q=None), "INVALID_ARG"),
                     (dict(k=None), "INVALID_ARG"), (dict(qo=None), "INVALID_ARG"), (dict(ko=ODD), "ALIGNMENT"),
                     (dict(q=ODD), "ALIGNMENT"), (dict(qs=511), "SHAPE"), (dict(qs=514), "ALIGNMENT"),
                     (dict(xt=1, qs=516), "ALIGNMENT"), (dict(ks=255), "SHAPE"), (dict(qos=500), "SHAPE"),
                     (dict(kos=258), "ALIGNMENT"), (dict(inv_freq=None), "INVALID_ARG"), (dict(inv_freq=ODD), "ALIGNMENT"),
                     (dict(pos=None), "INVALID_ARG"), (dict(pos=FAKE + 2), "ALIGNMENT"), (dict(q_weight=ODD), "ALIGNMENT"),
                     (dict(k_weight=ODD), "ALIGNMENT"), (dict(qo=FAKE, yt=1), "INVALID_ARG"),
                     (dict(qo=FAKE, qos=1024), "INVALID_ARG")]:
        assert _turn(**kw) == "MD_ERR_" + want, kw
    assert _turn(rows=0, q=None, k=None, qo=None, ko=None, pos=None, inv_freq=None) == "MD_OK"


def _routing(**kw):
    d = dict(k=4, score=1, groups=8, groups_kept=2, best_two=1, renorm=1, scale=1.0, balance=FAKE)
    d.update(kw)
    return ctypes.byref(md.RoutingDesc(*[d[n] for n, _ in md.RoutingDesc._fields_]))


def test_routing_refusals():
    L, sz = md.lib(), ctypes.c_size_t(0)
    size = L.md_moe_route_workspace_size
    for args, want in [((-1, 256, 64), "SHAPE"), ((4, 0, 64), "SHAPE"), ((4, 256, 0), "SHAPE"), ((4, 250, 64), "UNSUPPORTED"),
                       ((4, 16640, 64), "UNSUPPORTED"), ((4, 256, 257), "UNSUPPORTED"),
                       (((1 << 20) + 1, 256, 64), "UNSUPPORTED")]:
        assert _st(size(*args, ctypes.byref(sz))) == "MD_ERR_" + want, args
    assert _st(size(4, 256, 64, None)) == "MD_ERR_INVALID_ARG"
    assert size(0, 256, 64, ctypes.byref(sz)) == 0 and sz.value == 0
    assert size(100, 256, 64, ctypes.byref(sz)) == 0 and sz.value > 0

    def call(x=FAKE, xt=0, T=100, W=FAKE, bias=FAKE, idx=OUT, gates=OUT, logits=None, ws=FAKE, wsb=sz.value, r=None, **kw):
        return _st(L.md_moe_route(_routing(**kw) if r is None else r, x, xt, T, 256, W, bias, 64, idx, gates, logits, ws, wsb,
                                  None))
    for kw, want in [(dict(score=2), "INVALID_ARG"), (dict(best_two=2), "INVALID_ARG"), (dict(renorm=-1), "INVALID_ARG"),
                     (dict(scale=float("inf")), "INVALID_ARG"), (dict(k=0), "SHAPE"), (dict(k=65), "SHAPE"),
                     (dict(k=9), "UNSUPPORTED"), (dict(groups=0), "SHAPE"), (dict(groups=7), "SHAPE"),
                     (dict(groups_kept=0), "SHAPE"), (dict(groups_kept=9), "SHAPE"),
                     (dict(groups=32, groups_kept=1), "SHAPE"), (dict(groups=64, groups_kept=8), "SHAPE"),
                     (dict(balance=ODD), "ALIGNMENT"), (dict(xt=3), "INVALID_ARG"), (dict(x=None), "INVALID_ARG"),
                     (dict(W=None), "INVALID_ARG"), (dict(idx=None), "INVALID_ARG"), (dict(gates=None), "INVALID_ARG"),
                     (dict(x=ODD), "ALIGNMENT"), (dict(bias=ODD), "ALIGNMENT"), (dict(logits=ODD), "ALIGNMENT"),
                     (dict(ws=None), "WORKSPACE"), (dict(wsb=sz.value - 1), "WORKSPACE"), (dict(ws=ODD), "ALIGNMENT")]:
        assert call(**kw) == "MD_ERR_" + want, kw
    assert call(T=0, x=None, idx=None, gates=None, ws=None) == "MD_OK"
    assert _st(L.md_moe_route(None, FAKE, 0, 4, 256, FAKE, None, 64, OUT, OUT, None, FAKE, 1 << 30, None)) == \
        "MD_ERR_INVALID_ARG"


def test_routed_layer_refusals():
    L, sz = md.lib(), ctypes.c_size_t(0)
    m = md.MoELayerDesc(256, 256, 64, 4, 0, md.Q8_0, FAKE, FAKE, FAKE, None, None, None, FAKE, None, 0)
    ref = ctypes.byref(m)
    assert _st(L.md_moe_routed_workspace_size(None, 4, ctypes.byref(sz))) == "MD_ERR_INVALID_ARG"
    assert _st(L.md_moe_routed_workspace_size(ref, 129, ctypes.byref(sz))) == "MD_ERR_UNSUPPORTED"
    assert L.md_moe_routed_workspace_size(ref, 4, ctypes.byref(sz)) == 0 and sz.value > 0
    call = L.md_moe_layer_forward_routed
    assert _st(call(ref, _routing(k=3), FAKE, 4, OUT, None, None, FAKE, sz.value, None)) == "MD_ERR_SHAPE"
    assert _st(call(ref, None, FAKE, 4, OUT, None, None, FAKE, sz.value, None)) == "MD_ERR_INVALID_ARG"
    assert _st(call(ref, _routing(), FAKE, 4, None, None, None, FAKE, sz.value, None)) == "MD_ERR_INVALID_ARG"
    assert _st(call(ref, _routing(), ODD, 4, OUT, None, None, FAKE, sz.value, None)) == "MD_ERR_ALIGNMENT"
    assert _st(call(ref, _routing(), FAKE, 4, OUT, ODD, None, FAKE, sz.value, None)) == "MD_ERR_ALIGNMENT"
    assert _st(call(ref, _routing(), FAKE, 4, OUT, None, None, FAKE, sz.value - 1, None)) == "MD_ERR_WORKSPACE"
    assert _st(call(ref, _routing(), FAKE, 4, OUT, None, None, ODD, sz.value, None)) == "MD_ERR_ALIGNMENT"


def test_logprob_refusals():
    L, sz = md.lib(), ctypes.c_size_t(0)
    size = L.md_token_logprobs_workspace_size
    for args, want in [((-1, 100, 0), "SHAPE"), ((4, 0, 0), "SHAPE"), ((4, 100, -1), "SHAPE"), ((4, 5, 6), "SHAPE"),
                       (((1 << 20) + 1, 100, 0), "UNSUPPORTED"), ((4, (1 << 20) + 1, 0), "UNSUPPORTED"),
                       ((4, 100, 33), "UNSUPPORTED")]:
        assert _st(size(*args, ctypes.byref(sz))) == "MD_ERR_" + want, args
    assert _st(size(4, 100, 0, None)) == "MD_ERR_INVALID_ARG"
    assert size(4, 100, 8, ctypes.byref(sz)) == 0 and sz.value == 0       # one chunk: no workspace
    assert size(4, 100000, 8, ctypes.byref(sz)) == 0 and sz.value > 0

    def call(x=FAKE, xt=0, stride=100000, rows=4, V=100000, tok=FAKE, n=2, scale=1.0, top=8, lp=OUT, ent=OUT, ids=OUT,
             tlp=OUT, ws=FAKE, wsb=sz.value):
        return _st(L.md_token_logprobs(x, xt, stride, rows, V, tok, n, scale, top, lp, ent, ids, tlp, ws, wsb, None))
    for kw, want in [(dict(xt=2), "INVALID_ARG"), (dict(scale=0.0), "INVALID_ARG"), (dict(scale=float("nan")), "INVALID_ARG"),
                     (dict(scale=-1.0), "INVALID_ARG"), (dict(scale=3e38), "INVALID_ARG"), (dict(n=-1), "SHAPE"), (dict(n=65), "UNSUPPORTED"),
                     (dict(stride=99999), "SHAPE"), (dict(x=None), "INVALID_ARG"), (dict(tok=None), "INVALID_ARG"),
                     (dict(lp=None), "INVALID_ARG"), (dict(ids=None), "INVALID_ARG"), (dict(tlp=None), "INVALID_ARG"),
                     (dict(x=FAKE + 2), "ALIGNMENT"), (dict(xt=1, x=FAKE + 1), "ALIGNMENT"), (dict(tok=FAKE + 2), "ALIGNMENT"),
                     (dict(ent=OUT + 1), "ALIGNMENT"), (dict(ids=OUT + 2), "ALIGNMENT"), (dict(ws=None), "WORKSPACE"),
                     (dict(wsb=sz.value - 1), "WORKSPACE"), (dict(ws=ODD), "ALIGNMENT")]:
        assert call(**kw) == "MD_ERR_" + want, kw
    assert call(rows=0, x=None, tok=None, lp=None, ids=None, tlp=None, ent=None, ws=None) == "MD_OK"


def _mask(window=0, sinks=0, words=1, tree=FAKE):
    return ctypes.byref(md.KVMaskDesc(window, sinks, words, tree))


@pytest.mark.parametrize("kw,want", BAD_CACHE)
def test_masked_attention_bad_caches(kw, want):
    sz = ctypes.c_size_t(0)
    assert _st(md.lib().md_kv_attention_masked_workspace_size(ctypes.byref(_c(**kw)), ctypes.byref(_b()), 4, _mask(), 0,
                                                              ctypes.byref(sz))) == want


@pytest.mark.parametrize("kw,want", BAD_BATCH)
def test_masked_attention_bad_batches(kw, want):
    assert _st(md.lib().md_kv_attention_masked(ctypes.byref(_c()), ctypes.byref(_b(**kw)), FAKE, 0, 4, 512, 0.1, _mask(), OUT,
                                               0, 512, FAKE, 1 << 40, None)) == want


def test_masked_attention_refusals():
    L, sz = md.lib(), ctypes.c_size_t(0)
    c, b = ctypes.byref(_c()), ctypes.byref(_b(max_q=65))

    def att(q=FAKE, xt=0, heads=4, qs=512, scale=0.1, mask=None, out=OUT, yt=0, os_=512, ws=FAKE, wsb=1 << 40, bb=b):
        return _st(L.md_kv_attention_masked(c, bb, q, xt, heads, qs, scale, mask or _mask(words=2), out, yt, os_, ws, wsb, None))
    assert _st(L.md_kv_attention_masked(c, b, FAKE, 0, 4, 512, 0.1, None, OUT, 0, 512, FAKE, 1 << 40, None)) == \
        "MD_ERR_INVALID_ARG"
    for kw, want in [(dict(mask=_mask(sinks=-1, words=2)), "INVALID_ARG"), (dict(mask=_mask(window=-1, words=2)), "INVALID_ARG"),
                     (dict(mask=_mask(words=0)), "SHAPE"), (dict(mask=_mask(words=1)), "SHAPE"),
                     (dict(mask=_mask(words=16385)), "UNSUPPORTED"), (dict(mask=_mask(words=2, tree=FAKE + 4)), "ALIGNMENT"),
                     (dict(heads=3), "SHAPE"), (dict(heads=1026), "UNSUPPORTED"), (dict(xt=2), "INVALID_ARG"),
                     (dict(yt=2), "INVALID_ARG"), (dict(scale=float("nan")), "INVALID_ARG"), (dict(q=None), "INVALID_ARG"),
                     (dict(q=ODD), "ALIGNMENT"), (dict(qs=511), "SHAPE"), (dict(out=FAKE), "INVALID_ARG"),
                     (dict(os_=514), "ALIGNMENT")]:
        assert att(**kw) == "MD_ERR_" + want, kw
    wide = ctypes.byref(_b(S=1, max_kv=100000, stride=1563))
    m = _mask(window=50000, sinks=7, tree=None, words=0)
    assert L.md_kv_attention_masked_workspace_size(c, wide, 4, m, 0, ctypes.byref(sz)) == 0 and sz.value > 0
    assert att(bb=wide, mask=m, wsb=sz.value - 1) == "MD_ERR_WORKSPACE"
    assert _st(L.md_kv_attention_masked_workspace_size(c, wide, 4, m, 0, None)) == "MD_ERR_INVALID_ARG"
    none = ctypes.byref(_b(rows=0, q_start=None, kv_len=None, table=None))
    assert L.md_kv_attention_masked(c, none, None, 0, 4, 512, 0.1, m, None, 0, 512, None, 0, None) == 0


def test_tree_refusals():
    L = md.lib()

    def tree(par=FAKE, masks=OUT, words=1, pos=OUT, **kw):
        return _st(L.md_kv_tree(ctypes.byref(_b(**kw)), par, masks, words, pos, None))
    assert _st(L.md_kv_tree(None, FAKE, OUT, 1, OUT, None)) == "MD_ERR_INVALID_ARG"
    for kw, want in [(dict(S=0), "SHAPE"), (dict(rows=-1), "SHAPE"), (dict(max_q=0), "SHAPE"), (dict(S=65536), "UNSUPPORTED"),
                     (dict(max_q=1025, words=17), "UNSUPPORTED"), (dict(max_q=65), "SHAPE"), (dict(words=0), "SHAPE"),
                     (dict(words=16385), "UNSUPPORTED"), (dict(par=None), "INVALID_ARG"), (dict(masks=None), "INVALID_ARG"),
                     (dict(q_start=None), "INVALID_ARG"), (dict(kv_len=None), "INVALID_ARG"),
                     (dict(masks=OUT + 4), "ALIGNMENT"), (dict(par=FAKE + 2), "ALIGNMENT"), (dict(pos=OUT + 1), "ALIGNMENT")]:
        assert tree(**kw) == "MD_ERR_" + want, kw
    assert tree(rows=0, par=None, masks=None) == "MD_OK"


def test_binding_refusals():
    """What the C calls cannot see: types, shapes, layouts, and tensors of the CPU."""
    z = torch.zeros
    q, k, pos, inv = z(3, 4, 64), z(3, 2, 64), z(3, dtype=torch.int32), z(32)
    for args in [(z(3, 256), k, pos, inv), (q, z(2, 2, 64), pos, inv), (q, k.bfloat16(), pos, inv), (q, k, pos.long(), inv),
                 (q, k, pos[:2], inv), (q, k, pos, inv.double()), (q.transpose(1, 2), k, pos, inv), (q, k, pos, inv)]:
        with pytest.raises(ValueError):
            md.qk_norm_rope(*args)
    with pytest.raises(ValueError):
        md.qk_norm_rope(q, k, pos, inv, q_weight=z(63))
    r = md.Routing(2, balance=z(8))
    for x, W in [(z(3, 256).double().t().t()[:, ::2], z(8, 256)), (z(3, 256), z(8, 128)), (z(3, 256), z(8, 256).double()),
                 (z(3, 256), z(8, 256))]:
        with pytest.raises((ValueError, TypeError)):
            md.moe_route(x, W, r)
    with pytest.raises(ValueError):
        r.desc(9, torch.device("cpu"))
    for x, tok in [(z(3, 10).t(), None), (z(30), None), (z(3, 10), z(3, 1)), (z(3, 10), z(2, 1, dtype=torch.int32)),
                   (z(3, 10), z(3, dtype=torch.int32)), (z(3, 10), None)]:
        with pytest.raises(ValueError):
            md.token_logprobs(x, tokens=tok)
    c, b = streams._cache(), streams._batch()
    for kw in [dict(causal=False, sinks=2), dict(tree=z(3, 1)), dict(tree=z(2, 1, dtype=torch.int64)),
               dict(tree=z(3, dtype=torch.int64))]:
        with pytest.raises(ValueError):
            md.kv_attention(c, b, z(3, 4, 64), **kw)
    with pytest.raises(ValueError):
        md.kv_tree(b, z(3))
    with pytest.raises(ValueError):
        md.moe_layer_forward(streams._moe(), streams.X, routing=r, residual=streams.X)
