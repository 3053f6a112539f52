"""CPU checks of the 8-bit products' and the paged cache's entry points: every
bad argument is rejected with the documented status before anything is
enqueued (no call here reaches the GPU)."""
import ctypes

import pytest

import moe_decode_amd as md

FAKE = 0x7F0000000000
ODD = FAKE + 4


def _st(rc):
    return md.STATUS[rc]


def _w(type_=md.I8_ROW, rows=64, cols=256, q=FAKE, scale=FAKE):
    return ctypes.byref(md.QMatrixDesc(type_, rows, cols, q, scale))


def test_i8_errors():
    L = md.lib()
    sz = ctypes.c_size_t(0)
    qz = L.md_i8_quantize
    assert _st(qz(FAKE, 2, 4, 256, FAKE, FAKE, None)) == "MD_ERR_INVALID_ARG"
    assert _st(qz(FAKE, 0, -1, 256, FAKE, FAKE, None)) == "MD_ERR_SHAPE"
    assert _st(qz(FAKE, 0, 4, 0, FAKE, FAKE, None)) == "MD_ERR_SHAPE"
    assert _st(qz(FAKE, 0, 4, 255, FAKE, FAKE, None)) == "MD_ERR_UNSUPPORTED"
    assert _st(qz(FAKE, 0, 4, 16640, FAKE, FAKE, None)) == "MD_ERR_UNSUPPORTED"
    assert _st(qz(FAKE, 0, (1 << 20) + 1, 256, FAKE, FAKE, None)) == "MD_ERR_UNSUPPORTED"
    assert _st(qz(None, 0, 4, 256, FAKE, FAKE, None)) == "MD_ERR_INVALID_ARG"
    assert _st(qz(FAKE, 0, 4, 256, ODD, FAKE, None)) == "MD_ERR_ALIGNMENT"
    assert qz(None, 0, 0, 256, None, None, None) == 0          # no tokens: nothing to do
    mm = L.md_i8_matmul
    assert _st(mm(None, FAKE, FAKE, 4, None, FAKE, 0, None)) == "MD_ERR_INVALID_ARG"
    assert _st(mm(_w(type_=md.Q8_0), FAKE, FAKE, 4, None, FAKE, 0, None)) == "MD_ERR_UNSUPPORTED"
    assert _st(mm(_w(type_=md.I4_ROW), FAKE, FAKE, 4, None, FAKE, 0, None)) == "MD_ERR_UNSUPPORTED"
    assert _st(mm(_w(scale=None), FAKE, FAKE, 4, None, FAKE, 0, None)) == "MD_ERR_INVALID_ARG"
    assert _st(mm(_w(cols=250), FAKE, FAKE, 4, None, FAKE, 0, None)) == "MD_ERR_UNSUPPORTED"
    assert _st(mm(_w(), FAKE, FAKE, 4, None, FAKE, 3, None)) == "MD_ERR_INVALID_ARG"
    assert _st(mm(_w(), FAKE, None, 4, None, FAKE, 0, None)) == "MD_ERR_INVALID_ARG"
    assert _st(mm(_w(), FAKE, FAKE, 4, ODD, FAKE, 0, None)) == "MD_ERR_ALIGNMENT"
    assert _st(mm(_w(), FAKE, FAKE, -4, None, FAKE, 0, None)) == "MD_ERR_SHAPE"
    assert mm(_w(), None, None, 0, None, None, 0, None) == 0
    ws, lin = L.md_i8_linear_workspace_size, L.md_i8_linear
    assert _st(ws(_w(), 4, None)) == "MD_ERR_INVALID_ARG"
    assert ws(_w(), 0, ctypes.byref(sz)) == 0 and sz.value == 0
    assert ws(_w(), 5, ctypes.byref(sz)) == 0 and sz.value == 0          # the codes stay in the workgroups
    assert ws(_w(), 17, ctypes.byref(sz)) == 0 and sz.value == 17 * 256 + 256
    assert _st(lin(_w(), FAKE, 0, 17, None, FAKE, 0, FAKE, sz.value - 1, None)) == "MD_ERR_WORKSPACE"
    assert _st(lin(_w(), FAKE, 0, 17, None, FAKE, 0, None, sz.value, None)) == "MD_ERR_WORKSPACE"
    assert _st(lin(_w(), FAKE, 0, 17, None, FAKE, 0, ODD, sz.value, None)) == "MD_ERR_ALIGNMENT"
    assert _st(lin(_w(), FAKE, 5, 17, None, FAKE, 0, FAKE, sz.value, None)) == "MD_ERR_INVALID_ARG"
    assert _st(lin(_w(), None, 0, 17, None, FAKE, 0, FAKE, sz.value, None)) == "MD_ERR_INVALID_ARG"


def _c(n=8, page=64, heads=2, dim=128, k=FAKE, v=FAKE, ks=FAKE, vs=FAKE):
    return md.KVCacheDesc(n, page, heads, dim, k, v, ks, vs)


def _b(S=3, rows=3, max_q=1, max_kv=100, stride=2, q_start=FAKE, kv_len=FAKE, table=FAKE):
    return md.KVBatchDesc(S, rows, max_q, max_kv, stride, q_start, kv_len, table)


BAD_CACHE = [(dict(n=0), "MD_ERR_SHAPE"), (dict(heads=0), "MD_ERR_SHAPE"), (dict(heads=257), "MD_ERR_UNSUPPORTED"),
             (dict(dim=96), "MD_ERR_UNSUPPORTED"), (dict(page=32), "MD_ERR_UNSUPPORTED"),
             (dict(page=100), "MD_ERR_UNSUPPORTED"), (dict(k=None), "MD_ERR_INVALID_ARG"),
             (dict(v=ODD), "MD_ERR_ALIGNMENT"), (dict(ks=None), "MD_ERR_INVALID_ARG"), (dict(vs=ODD), "MD_ERR_ALIGNMENT")]
BAD_BATCH = [(dict(S=0), "MD_ERR_SHAPE"), (dict(S=65536), "MD_ERR_UNSUPPORTED"), (dict(rows=-1), "MD_ERR_SHAPE"),
             (dict(max_q=0), "MD_ERR_SHAPE"), (dict(max_kv=0), "MD_ERR_SHAPE"), (dict(max_kv=129), "MD_ERR_SHAPE"),
             (dict(max_kv=(1 << 30) + 1, stride=1 << 25), "MD_ERR_UNSUPPORTED"),
             (dict(stride=0), "MD_ERR_SHAPE"), (dict(rows=(1 << 20) + 1), "MD_ERR_UNSUPPORTED"),
             (dict(q_start=None), "MD_ERR_INVALID_ARG"), (dict(kv_len=FAKE + 2), "MD_ERR_ALIGNMENT"),
             (dict(table=None), "MD_ERR_INVALID_ARG")]


@pytest.mark.parametrize("kw,want", BAD_CACHE)
def test_bad_caches(kw, want):
    L, sz, n = md.lib(), ctypes.c_size_t(0), (ctypes.c_int32 * 1)(0)
    c, b = ctypes.byref(_c(**kw)), ctypes.byref(_b())
    assert _st(L.md_kv_append(c, b, FAKE, 256, FAKE, 256, 0, None)) == want
    assert _st(L.md_kv_attention_workspace_size(c, b, 4, 1, 0, 0, ctypes.byref(sz))) == want
    assert _st(L.md_kv_read_pages(c, FAKE, 1, FAKE, FAKE, 0, None)) == want
    assert _st(L.md_kv_copy_pages(c, n, n, 1, None)) == want


@pytest.mark.parametrize("kw,want", BAD_BATCH)
def test_bad_batches(kw, want):
    L = md.lib()
    c, b = ctypes.byref(_c()), ctypes.byref(_b(**kw))
    assert _st(L.md_kv_append(c, b, FAKE, 256, FAKE, 256, 0, None)) == want
    assert _st(L.md_kv_attention(c, b, FAKE, 0, 4, 512, 0.1, 1, 0, FAKE, 0, 512, FAKE, 1 << 40, None)) == want


def test_attention_and_append_errors():
    L, sz = md.lib(), ctypes.c_size_t(0)
    c, b = ctypes.byref(_c()), ctypes.byref(_b())

    def att(q=FAKE, xt=0, heads=4, qs=512, scale=0.1, causal=1, window=0, out=FAKE + 65536, yt=0, os_=512, ws=FAKE,
            wsb=1 << 40, bb=b):
        return _st(L.md_kv_attention(c, bb, q, xt, heads, qs, scale, causal, window, out, yt, os_, ws, wsb, None))
    assert att(heads=3) == "MD_ERR_SHAPE"
    assert att(heads=0) == "MD_ERR_SHAPE"
    assert att(heads=1026) == "MD_ERR_UNSUPPORTED"
    assert att(causal=2) == "MD_ERR_INVALID_ARG"
    assert att(window=-1) == "MD_ERR_INVALID_ARG"
    assert att(window=5, causal=0) == "MD_ERR_INVALID_ARG"
    assert att(xt=2) == "MD_ERR_INVALID_ARG"
    assert att(yt=-1) == "MD_ERR_INVALID_ARG"
    assert att(scale=float("nan")) == "MD_ERR_INVALID_ARG"
    assert att(scale=float("inf")) == "MD_ERR_INVALID_ARG"
    assert att(q=None) == "MD_ERR_INVALID_ARG"
    assert att(q=ODD) == "MD_ERR_ALIGNMENT"
    assert att(qs=511) == "MD_ERR_SHAPE"
    assert att(qs=514) == "MD_ERR_ALIGNMENT"
    assert att(xt=1, qs=516) == "MD_ERR_ALIGNMENT"
    assert att(out=FAKE) == "MD_ERR_INVALID_ARG"        # in place
    assert att(os_=500) == "MD_ERR_SHAPE"
    wide = ctypes.byref(_b(S=1, max_kv=100000, stride=1563))
    assert L.md_kv_attention_workspace_size(c, wide, 4, 1, 0, 0, ctypes.byref(sz)) == 0 and sz.value > 0
    assert att(bb=wide, wsb=sz.value - 1) == "MD_ERR_WORKSPACE"
    assert att(bb=wide, ws=None) == "MD_ERR_WORKSPACE"
    assert att(bb=wide, ws=ODD) == "MD_ERR_ALIGNMENT"
    assert _st(L.md_kv_attention_workspace_size(c, wide, 4, 1, 0, 0, None)) == "MD_ERR_INVALID_ARG"
    assert _st(L.md_kv_attention_workspace_size(c, wide, 4, 1, 0, 2, ctypes.byref(sz))) == "MD_ERR_INVALID_ARG"
    none = ctypes.byref(_b(rows=0, q_start=None, kv_len=None, table=None))
    assert L.md_kv_attention(c, none, None, 0, 4, 512, 0.1, 1, 0, None, 0, 512, None, 0, None) == 0
    assert L.md_kv_append(c, none, None, 256, None, 256, 0, None) == 0
    ap = L.md_kv_append
    assert _st(ap(c, b, FAKE, 255, FAKE, 256, 0, None)) == "MD_ERR_SHAPE"
    assert _st(ap(c, b, FAKE, 256, FAKE, 258, 0, None)) == "MD_ERR_ALIGNMENT"
    assert _st(ap(c, b, FAKE, 256, FAKE, 260, 1, None)) == "MD_ERR_ALIGNMENT"
    assert _st(ap(c, b, None, 256, FAKE, 256, 0, None)) == "MD_ERR_INVALID_ARG"
    assert _st(ap(c, b, FAKE, 256, FAKE, 256, 7, None)) == "MD_ERR_INVALID_ARG"
    rd = L.md_kv_read_pages
    assert _st(rd(c, FAKE, 1 << 24, FAKE, FAKE, 0, None)) == "MD_ERR_UNSUPPORTED"
    assert _st(rd(c, None, 2, FAKE, FAKE, 0, None)) == "MD_ERR_INVALID_ARG"
    assert _st(rd(c, FAKE + 2, 2, FAKE, FAKE, 0, None)) == "MD_ERR_ALIGNMENT"
    assert _st(rd(c, FAKE, -2, FAKE, FAKE, 0, None)) == "MD_ERR_SHAPE"
    assert _st(rd(c, FAKE, 2, FAKE, None, 0, None)) == "MD_ERR_INVALID_ARG"
    assert rd(c, None, 0, None, None, 0, None) == 0


@pytest.mark.parametrize("src,dst", [([0], [8]), ([-1], [3]), ([1], [1]), ([1, 2], [3, 3]), ([1, 3], [3, 4]),
                                     ([1, 4], [4, 2])])
def test_copy_pairs_that_meet_are_refused(src, dst):
    L, n = md.lib(), len(src)
    c = ctypes.byref(_c())
    a = ctypes.c_int32 * n
    assert _st(L.md_kv_copy_pages(c, a(*src), a(*dst), n, None)) == "MD_ERR_INVALID_ARG"
    assert _st(L.md_kv_copy_pages(c, None, a(*dst), n, None)) == "MD_ERR_INVALID_ARG"
    assert _st(L.md_kv_copy_pages(c, a(*src), a(*dst), -1, None)) == "MD_ERR_SHAPE"
    assert L.md_kv_copy_pages(c, None, None, 0, None) == 0


def test_matrices_that_do_not_hold_what_they_say():
    """The binding refuses what the C call cannot see: a matrix on another
    device than the call's tensors, too short, or with scales of another type."""
    import torch
    q, s = torch.zeros(64 * 256, dtype=torch.int8), torch.zeros(64)
    ok = md.DevQMatrix("i8_row", 64, 256, q, s)
    md._i8_desc(ok, torch.device("cpu"))
    with pytest.raises(ValueError):
        md._i8_desc(ok, torch.device("cuda:0"))
    for bad in (md.DevQMatrix("i8_row", 64, 512, q, s), md.DevQMatrix("i8_row", 64, 256, q, s.double()),
                md.DevQMatrix("i8_row", 64, 256, q, s[:63]), md.DevQMatrix("i8_row", 64, 256, q.view(64, 256).t(), s)):
        with pytest.raises(ValueError):
            md._i8_desc(bad, torch.device("cpu"))
