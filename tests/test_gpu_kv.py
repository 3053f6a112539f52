"""The paged 8-bit cache on the GPU: appends equal to the model's codes and
scales, attention within the derived bound of the definition in 64 bits on the
codes the cache holds, page reads and copies exact; and a decoder layer made of
them, eager and captured."""
import numpy as np
import pytest

from .gpu_common import require_gpu, say
from .kv_model import Cache, attention, many_columns

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _i32(v):
    import torch
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def _to_gpu(m):
    """The model's cache as the library's."""
    import moe_decode_amd as md
    import torch
    return md.KVCache(torch.from_numpy(m.c["k"]).cuda().contiguous(),
                      torch.from_numpy(m.c["v"]).cuda().transpose(2, 3).contiguous(),
                      torch.from_numpy(m.s["k"]).cuda(), torch.from_numpy(m.s["v"]).cuda())


def _from_gpu(c, m):
    m.c = {"k": c.k.cpu().numpy().copy(), "v": c.v.cpu().numpy().transpose(0, 1, 3, 2).copy()}
    m.s = {"k": c.k_scale.cpu().numpy().copy(), "v": c.v_scale.cpu().numpy().copy()}


def _batch(nq, lens, table, max_q=None, max_kv=None):
    import moe_decode_amd as md
    starts = np.concatenate([[0], np.cumsum(nq)])
    return md.KVBatch(_i32(starts), _i32(lens), _i32(table), max_q or max(max(nq), 1), max_kv or max(max(lens), 1))


def _tables(lens, page, rng, spare=0):
    need = [-(-n // page) for n in lens]
    order = rng.permutation(sum(need) + spare)
    t, at = np.full((len(lens), max(max(need), 1)), -1, np.int32), 0
    for i, n in enumerate(need):
        t[i, :n] = order[at:at + n]
        at += n
    return t, sum(need) + spare


def _rn(rng, shape, xt):
    import torch
    x = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda().to(_dt(xt))
    return x, x.float().cpu().numpy()


# ---- append ----------------------------------------------------------------

APPENDS = [  # heads, dim, page, (new, length) of each sequence
    (1, 64, 64, [(1, 1)]),
    (2, 128, 64, [(1, 64), (1, 65), (1, 100), (0, 70), (3, 66)]),
    (3, 64, 128, [(130, 200), (128, 256), (1, 129), (129, 129)]),
    (2, 256, 64, [(65, 128), (2, 130), (64, 127)]),
    (1, 128, 256, [(257, 300), (256, 256), (1, 512), (17, 33)]),
    (2, 64, 64, [(1, 2), (1, 6), (1, 7), (1, 8), (2, 70), (1, 64)]),      # every place in a word, held tokens before it
    (1, 256, 256, [(3, 35), (8, 30), (1, 131)]),
    (1, 256, 256, [(256, 256), (300, 400), (1, 700)]),                     # whole pages of 64 KB
]


@pytest.mark.parametrize("heads,dim,page,seqs", APPENDS)
@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_append_gives_the_models_codes(heads, dim, page, seqs, xt):
    import moe_decode_amd as md
    import torch
    rng = np.random.default_rng(heads * dim + page)
    nq, lens = [a for a, _ in seqs], [b for _, b in seqs]
    table, n = _tables(lens, page, rng, spare=2)
    m = Cache(n, heads, page, dim, rng)
    c = _to_gpu(m)
    rows = sum(nq)
    (k, kn), (v, vn) = _rn(rng, (rows, heads, dim), xt), _rn(rng, (rows, heads, dim), xt)
    k[::3] *= 4.0       # some raise their page's scale, by more than once
    kn[::3] *= 4.0
    md.kv_append(c, _batch(nq, lens, np.maximum(table, 0)), k, v)
    at = 0
    for i, (a, b) in enumerate(seqs):
        m.append(table[i], b - a, {"k": kn[at:at + a], "v": vn[at:at + a]})
        at += a
    g = Cache(n, heads, page, dim, rng)
    _from_gpu(c, g)
    for name in "kv":
        assert np.array_equal(g.s[name], m.s[name]), name
        assert np.array_equal(g.c[name], m.c[name]), (name, np.argwhere(g.c[name] != m.c[name])[:4].tolist())
    # the same, read back as values
    k2, v2 = md.kv_read_pages(c, _i32(range(n)))
    assert np.array_equal(k2.cpu().numpy(), m.c["k"] * m.s["k"][..., None, None])
    assert np.array_equal(v2.cpu().numpy(), m.c["v"] * m.s["v"][..., None, None])
    kb, vb = md.kv_read_pages(c, _i32([n - 1, 0, n - 1]), out_dtype=torch.bfloat16)
    pick = [n - 1, 0, n - 1]
    assert torch.equal(kb, k2[pick].bfloat16()) and torch.equal(vb, v2[pick].bfloat16())


def test_token_by_token_and_zero_rows():
    """A page filled one token at a time, growing values: the scale rises by
    powers of two and a held value stays within one step; zeros first (a scale
    of 0), tiny and subnormal values next."""
    import moe_decode_amd as md
    heads, dim, page = 2, 64, 64
    rng = np.random.default_rng(3)
    m = Cache(2, heads, page, dim, rng)
    c = _to_gpu(m)
    table = np.array([[1, 0]], np.int32)
    sizes = [0, 0, 1e-44, 3e-39, 1e-30, 1e-12] + [1.05 ** i for i in range(70)]
    said = []
    for t, size in enumerate(sizes):
        (k, kn), (v, vn) = _rn(rng, (1, heads, dim), "f32"), _rn(rng, (1, heads, dim), "f32")
        k, kn = k * np.float32(size), kn * np.float32(size)
        md.kv_append(c, _batch([1], [t + 1], table), k, v)
        m.append(table[0], t, {"k": kn, "v": vn})
        said.append((kn[0], vn[0]))
    g = Cache(2, heads, page, dim, rng)
    _from_gpu(c, g)
    for name in "kv":
        assert np.array_equal(g.s[name], m.s[name])
        assert np.array_equal(g.c[name], m.c[name])
        got = g.values(name, table[0], len(sizes))
        step = g.s[name][[1] * 64 + [0] * (len(sizes) - 64)].astype(np.float64)
        want = np.stack([s["kv".index(name)] for s in said]).astype(np.float64)
        assert (np.abs(got - want) <= step[:, :, None] * (1 + 1e-6)).all()


def test_append_leaves_alone_what_it_must():
    """Bad statements write nothing: a length past max_kv, a run past max_q, rows
    out of order, pages that are none; negative positions are left out; a
    non-finite value makes its page and head's scale NaN and no other's."""
    import moe_decode_amd as md
    import torch
    heads, dim, page = 2, 64, 64
    rng = np.random.default_rng(4)
    m = Cache(4, heads, page, dim, rng)
    (k, kn), (v, vn) = _rn(rng, (6, heads, dim), "f32"), _rn(rng, (6, heads, dim), "f32")

    def run(starts, lens, table, max_q=6, max_kv=128):
        c = _to_gpu(m)
        md.kv_append(c, md.KVBatch(_i32(starts), _i32(lens), _i32(table), max_q, max_kv), k, v)
        g = Cache(4, heads, page, dim, rng)
        _from_gpu(c, g)
        return g, [p for p in range(4) if any(not np.array_equal(g.c[n][p], m.c[n][p]) or
                                              not np.array_equal(g.s[n][p], m.s[n][p]) for n in "kv")]
    good = [[0, 1], [2, 3]]
    assert run([0, 3, 6], [70, 10], good)[1] == [1, 2]
    assert run([0, 3, 6], [129, 10], good)[1] == [2]
    assert run([0, 3, 6], [-1, 10], good)[1] == [2]
    assert run([0, 3, 6], [70, 10], good, max_q=2)[1] == []
    assert run([3, 0, 6], [70, 10], good)[1] == [2]
    assert run([0, 3, 7], [70, 10], good)[1] == [1]
    assert run([-1, 3, 6], [70, 10], good)[1] == [2]
    assert run([0, 3, 6], [70, 10], [[0, 4], [-1, 3]])[1] == []
    g, touched = run([0, 6, 6], [2, 10], good)      # four of six tokens lie before position 0
    assert touched == [0]
    e = Cache(4, heads, page, dim, np.random.default_rng(4))
    e.append([0], -4, {"k": kn, "v": vn})
    assert np.array_equal(g.c["k"][0][:, :2], e.c["k"][0][:, :2]) and np.array_equal(g.s["v"][0], e.s["v"][0])
    k[1, 1, 5], v[2, 0, 0] = float("inf"), float("nan")
    g, _ = run([0, 3, 6], [70, 10], good)
    assert np.isnan(g.s["k"][1, 1]) and np.isfinite(g.s["k"][1, 0]) and np.isnan(g.s["v"][1, 0])
    assert np.isfinite(g.s["k"][2]).all() and np.isfinite(g.s["v"][2]).all()


def test_strided_rows_of_a_joint_projection():
    import moe_decode_amd as md
    import torch
    heads, dim, page = 2, 64, 64
    rng = np.random.default_rng(5)
    (qkv, host) = _rn(rng, (5, 8 * dim), "bf16")
    k, v = qkv[:, 4 * dim:6 * dim].view(5, 2, dim), qkv[:, 6 * dim:].view(5, 2, dim)
    a, b = md.KVCache.empty(1, heads, dim, page), md.KVCache.empty(1, heads, dim, page)
    for c in (a, b):
        c.k.zero_(), c.v.zero_()
    bt = _batch([5], [5], [[0]])
    md.kv_append(a, bt, k, v)
    md.kv_append(b, bt, k.contiguous(), v.contiguous())
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v) and torch.equal(a.k_scale, b.k_scale)
    q = qkv[:, :4 * dim].view(5, 4, dim)
    out = torch.full((5, 3, 4, dim), 9.0, device="cuda")
    y = md.kv_attention(a, bt, q, out=out[:, 1])
    assert torch.equal(out[:, 1], md.kv_attention(a, bt, q.contiguous()))
    assert bool((out[:, 0] == 9.0).all()) and bool((out[:, 2] == 9.0).all()) and y.data_ptr() == out[:, 1].data_ptr()


# ---- attention ---------------------------------------------------------------

ATTN = [  # key heads, group, dim, page, (new, length) of each sequence, causal, window
    (1, 1, 64, 64, [(1, 1)], True, 0),
    (2, 4, 64, 64, [(1, 97), (1, 64), (1, 65), (1, 2)], True, 0),
    (4, 8, 64, 64, [(1, 200), (1, 63), (1, 128)], True, 0),
    (2, 8, 128, 64, [(1, 1000), (1, 1), (1, 513), (0, 10), (1, 640)], True, 0),
    (1, 16, 128, 128, [(1, 3000), (1, 129)], True, 0),
    (2, 3, 128, 128, [(7, 300), (1, 5), (40, 40), (17, 129)], True, 0),
    (1, 7, 256, 64, [(5, 77), (33, 100)], True, 0),
    (3, 1, 256, 256, [(1, 700), (3, 257)], True, 0),
    (2, 5, 64, 256, [(20, 400), (9, 64)], True, 33),
    (2, 2, 128, 64, [(70, 200), (1, 150)], True, 1),
    (1, 4, 256, 128, [(1, 900), (6, 500)], True, 300),
    (2, 2, 64, 64, [(3, 190), (50, 7), (1, 64)], False, 0),
    (1, 3, 128, 128, [(9, 260), (2, 0)], False, 0),
    (2, 4, 128, 64, [(5, 3), (4, 0), (3, 3)], True, 0),
    (1, 2, 64, 64, [(150, 150)], True, 0),
    (1, 4, 128, 64, [(130, 333)], True, 0),
    (1, 64, 64, 64, [(1, 100), (2, 70)], True, 0),
    (2, 4, 128, 64, [(40, 1500), (3, 50), (17, 17)], True, 0),
    (1, 16, 64, 128, [(4, 900), (5, 1000)], False, 0),
    (1, 5, 256, 64, [(13, 700), (20, 90)], True, 200),
    (1, 8, 256, 64, [(70, 700), (3, 90)], True, 0),
    (2, 4, 128, 64, [(12, 5), (5, 300)], True, 2 ** 31 - 1),                # windows past every position, and runs
    (1, 4, 64, 64, [(200, 90), (3, 64)], True, 2 ** 31 - 1),                # that begin before the first one
    (2, 4, 64, 64, [(9, 100), (2, 100)], True, 100),
    (1, 8, 256, 64, [(100, 700), (3, 90)], True, 0),
    (1, 8, 256, 128, [(110, 3000)], True, 500),
]


@pytest.mark.parametrize("case", range(len(ATTN)))
@pytest.mark.parametrize("xt,out", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
def test_attention(case, xt, out):
    import moe_decode_amd as md
    import torch
    Hkv, G, dim, page, seqs, causal, window = ATTN[case]
    say(f"[attn] {ATTN[case]} {xt} -> {out}")
    rng = np.random.default_rng(case)
    nq, lens = [a for a, _ in seqs], [b for _, b in seqs]
    table, n = _tables(lens, page, rng, spare=1)
    m = Cache(n, Hkv, page, dim, rng)
    c = _to_gpu(m)
    rows = sum(nq)
    q, qn = _rn(rng, (rows + 1, Hkv * G, dim), xt)
    y = torch.full((rows + 1, Hkv * G, dim), 5.0, dtype=_dt(out), device="cuda")
    scale = 2.0 / dim ** 0.5
    # the entries behind a sequence's pages name no page: they are not read
    md.kv_attention(c, _batch(nq, lens, table), q, scale=scale, causal=causal, window=window, out=y)
    got, at = y.double().cpu().numpy(), 0
    worst = 0.0
    for i, (a, b) in enumerate(seqs):
        want, tol = attention(qn[at:at + a], m.values("k", table[i], b), m.values("v", table[i], b), scale, causal,
                              window, out, many=many_columns(max(nq), G, dim, out))
        err = np.abs(got[at:at + a] - want)
        assert (err <= tol).all(), (i, float((err / tol).max()))
        worst = max(worst, float((err / np.maximum(tol, 1e-30)).max()) if a else 0.0)
        at += a
    say(f"  worst error / bound {worst:.3f}")
    assert bool((y[rows] == 5.0).all())     # the row behind the last sequence


@pytest.mark.parametrize("max_q", [4, 300])
def test_every_weight_is_right(max_q):
    """Values of which each channel holds one token: the outputs are the softmax
    weights, each within the bound by itself (4 rows of 4 heads: the form for
    few columns; 300 of them: the one for many, whose weights are two f16)."""
    import moe_decode_amd as md
    Hkv, G, dim, page = 1, 4, 64, 64
    rng = np.random.default_rng(77)
    m = Cache(1, Hkv, page, dim, rng)
    m.c["v"][:] = (127 * np.eye(64)).astype(np.int8)
    m.s["v"][:] = 1 / 127
    c = _to_gpu(m)
    q, qn = _rn(rng, (max_q, G, dim), "f32")
    q, qn = q * 0.25, qn * np.float32(0.25)
    y = md.kv_attention(c, _batch([max_q], [64], [[0]]), q, causal=False).double().cpu().numpy()
    want, tol = attention(qn, m.values("k", [0], 64), m.values("v", [0], 64), 0.125, False, 0, "f32", many=max_q > 16)
    assert (tol <= 1e-4 * want).all()
    assert (np.abs(y - want) <= tol).all(), float((np.abs(y - want) / want).max())


@pytest.mark.parametrize("S,Hkv,G,D,page,window,out", [
    (700, 1, 2, 64, 64, 0, "f32"), (1024, 1, 1, 64, 64, 0, "bf16"), (1025, 1, 1, 64, 64, 0, "f32"),
    (37, 2, 8, 128, 64, 0, "f32"), (37, 2, 8, 128, 128, 90, "bf16"), (5, 1, 3, 256, 256, 0, "f32"),
    (3, 4, 5, 64, 64, 700, "f32")])
def test_ragged_batches_dealt_out(S, Hkv, G, D, page, window, out):
    """Sequences of 0 to 4500 positions with 0 to 3 new rows each, some without
    rows, some that see nothing: every row against the definition; the same call
    again gives the same bits."""
    import moe_decode_amd as md
    import torch
    rng = np.random.default_rng(S + D)
    nq = rng.integers(0, 4, S)
    lens = np.where(rng.random(S) < 0.7, rng.integers(0, 40, S), rng.integers(0, 1500, S))
    nq[-1], lens[-1], nq[0], lens[1] = 0, 4500, 3, 4300
    nq, lens = nq.tolist(), lens.tolist()
    table, n = _tables(lens, page, rng)
    m = Cache(n, Hkv, page, D, rng)
    c = _to_gpu(m)
    q, qn = _rn(rng, (sum(nq) + 1, Hkv * G, D), "f32")
    b = _batch(nq, lens, table, max_q=3)
    y = torch.full((sum(nq) + 1, Hkv * G, D), 5.0, dtype=_dt(out), device="cuda")
    md.kv_attention(c, b, q, window=window, out=y)
    got, at = y.double().cpu().numpy(), 0
    for i, (a, L) in enumerate(zip(nq, lens)):
        if a:
            want, tol = attention(qn[at:at + a], m.values("k", table[i], L), m.values("v", table[i], L), D ** -0.5,
                                  True, window, out)
            assert (np.abs(got[at:at + a] - want) <= tol).all(), (i, a, L)
        at += a
    assert bool((y[-1] == 5.0).all())
    for _ in range(3):
        z = torch.full_like(y, 5.0)
        md.kv_attention(c, b, q, window=window, out=z)
        assert torch.equal(z, y)


def test_long_context_split_over_workgroups():
    """131072 + 3 positions (offsets of a page past 2^31 bytes are not reached
    here, but every split is), against the sum in 64 bits on the GPU."""
    import moe_decode_amd as md
    import torch
    Hkv, G, dim, page, L = 2, 4, 128, 64, 131075
    g = torch.Generator(device="cuda").manual_seed(1)
    n = -(-L // page)
    k = torch.randint(-127, 128, (n, Hkv, page, dim), generator=g, dtype=torch.int8, device="cuda")
    v = torch.randint(-127, 128, (n, Hkv, dim, page), generator=g, dtype=torch.int8, device="cuda")
    ks, vs = (0.005 + 0.02 * torch.rand(n, Hkv, generator=g, device="cuda") for _ in range(2))
    c = md.KVCache(k, v, ks, vs)
    perm = torch.randperm(n, generator=torch.Generator().manual_seed(2), dtype=torch.int32)
    q = torch.randn(1, Hkv * G, dim, generator=g, device="cuda")
    got = md.kv_attention(c, _batch([1], [L], perm.numpy()[None]), q).double()
    p = perm.long().cuda()
    for h in range(Hkv):
        kk = (k[p, h].double() * ks[p, h].double()[:, None, None]).reshape(-1, dim)[:L]
        vv = (v[p, h].double() * vs[p, h].double()[:, None, None]).transpose(1, 2).reshape(-1, dim)[:L]
        qq = q[0, h * G:(h + 1) * G].double()
        s = (qq @ kk.t().contiguous()) / dim ** 0.5
        e = torch.exp(s - s.amax(1, keepdim=True))
        w = e / e.sum(1, keepdim=True)
        want, V = w @ vv, w @ vv.abs()
        u, t = 2.0 ** -24, 8355711.0        # as in the model's bound
        A = (qq.abs().amax(1) * kk.abs().sum(1).max()) / dim ** 0.5
        ds = A * (0.5 / t + 2 * u) + 24 * u * s.abs().amax(1)
        tol = (2 * (ds + 4 * u + (2 * L / 64 + 40) * u))[:, None] * V + \
            (vv.abs().sum(0)[None] + L * V) / t / e.sum(1, keepdim=True)
        assert bool(((got[0, h * G:(h + 1) * G] - want).abs() <= 1.05 * tol).all())


def test_offsets_past_32_bits():
    """A cache of over 2^32 bytes of codes: its last page is written, read,
    attended and copied."""
    import moe_decode_amd as md
    import torch
    Hkv, dim, page = 8, 256, 256
    per = Hkv * dim * page
    n = (1 << 32) // per + 3
    c = md.KVCache.empty(n, Hkv, dim, page)
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v, q = (torch.randn(70, h, dim, generator=g, device="cuda") for h in (Hkv, Hkv, 2 * Hkv))
    small = md.KVCache.empty(2, Hkv, dim, page)
    md.kv_append(small, _batch([70], [70], [[1]]), k, v)
    md.kv_append(c, _batch([70], [70], [[n - 1]]), k, v)
    want = md.kv_attention(small, _batch([70], [70], [[1]]), q)
    assert torch.equal(md.kv_attention(c, _batch([70], [70], [[n - 1]]), q), want)
    md.kv_copy_pages(c, [n - 1], [n - 2])
    assert torch.equal(md.kv_attention(c, _batch([70], [70], [[n - 2]]), q), want)
    a, b = md.kv_read_pages(c, _i32([n - 1, n - 2])), md.kv_read_pages(small, _i32([1, 1]))
    assert torch.equal(a[0][:, :, :70], b[0][:, :, :70]) and torch.equal(a[1][:, :, :70], b[1][:, :, :70])


def test_values_that_are_not_finite_stay_with_their_rows():
    import moe_decode_amd as md
    import torch
    Hkv, G, dim, page = 2, 2, 64, 64
    rng = np.random.default_rng(8)
    lens = [200, 130]
    table, n = _tables(lens, page, rng)
    m = Cache(n, Hkv, page, dim, rng)
    m.s["k"][table[0, 2], 0] = np.nan          # positions 128..191, head 0
    m.s["v"][table[1, 0], 1] = np.inf          # positions 0..63, head 1
    c = _to_gpu(m)
    (q, qn) = _rn(rng, (130, Hkv * G, dim), "f32")
    q[129, 3, 7] = float("nan")                # the last row of the second sequence
    y = md.kv_attention(c, _batch([100, 30], lens, table), q).cpu().numpy()
    # rows of the first sequence: positions 100..199
    bad = np.zeros((130, Hkv * G), bool)
    bad[28:100, :2] = True
    bad[100:, 2:] = True
    assert np.array_equal(np.isnan(y).all(2), bad) and np.array_equal(np.isnan(y).any(2), bad)
    y = md.kv_attention(c, _batch([100, 30], lens, table), q, window=10).cpu().numpy()
    bad[:] = False
    bad[28:100, :2] = True                     # positions 128..199 still see 128..191 up to 200
    bad[28 + 64 + 9:100, :2] = False
    bad[129, 3] = True
    assert np.array_equal(np.isnan(y).any(2), bad)
    # pages that are none, and statements that do not hold
    y = md.kv_attention(c, _batch([100, 30], lens, np.where(table == table[0, 3], n, table)), q[:, :, :]).cpu().numpy()
    assert np.isnan(y[92:100]).all() and np.isfinite(y[:28]).all()
    b = _batch([100, 30], [200, 130], table, max_kv=150)
    y = md.kv_attention(c, b, q).cpu().numpy()
    assert np.isnan(y[:100]).all() and np.isfinite(y[100:, :2]).all()
    out = torch.full((130, Hkv * G, dim), 3.0, device="cuda")
    md.kv_attention(c, md.KVBatch(_i32([0, 131, 130]), _i32(lens), _i32(table), 100, 200), q, out=out)
    assert bool((out == 3.0).all())


def test_scales_far_apart_and_large_scores():
    """Scores of hundreds (a softmax of one key) and pages whose scales differ
    by 2^40: against the model."""
    import moe_decode_amd as md
    Hkv, G, dim, page = 1, 2, 64, 64
    rng = np.random.default_rng(12)
    lens = [300]
    table, n = _tables(lens, page, rng)
    m = Cache(n, Hkv, page, dim, rng)
    m.s["v"][:, 0] = np.exp2(rng.integers(-20, 20, n)).astype(np.float32)
    m.s["k"][:, 0] = 0.3
    c = _to_gpu(m)
    q, qn = _rn(rng, (4, G, dim), "f32")
    for scale in (4.0, -4.0, 0.0):
        for max_q in (4, 40):       # the forms for few and for many columns
            y = md.kv_attention(c, _batch([4], lens, table, max_q=max_q), q, scale=scale).double().cpu().numpy()
            want, tol = attention(qn, m.values("k", table[0], 300), m.values("v", table[0], 300), scale, True, 0,
                                  "f32", many=max_q == 40)
            assert (np.abs(y - want) <= tol).all()


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("grow", [0.3, 2.0, 30.0])
def test_maxima_that_grow(out, many, grow):
    """Keys that get larger from page to page, so that a row's largest score keeps
    rising by a little or a lot, and then smaller again."""
    import moe_decode_amd as md
    Hkv, G, dim, page, n = 2, 2, 64, 64, 12
    rng = np.random.default_rng(91)
    m = Cache(n, Hkv, page, dim, rng)
    up = np.minimum(np.arange(n), 16 - np.arange(n)) + 1
    m.s["k"][:] = (grow / 127 * up)[:, None].astype(np.float32)
    m.s["v"][:] = np.float32(0.01)
    c = _to_gpu(m)
    q, qn = _rn(rng, (5, Hkv * G, dim), "bf16")
    got = md.kv_attention(c, _batch([5], [n * page - 3], [list(range(n))], max_q=40 if many else 5), q, out_dtype=_dt(out))
    want, tol = attention(qn, m.values("k", range(n), n * page - 3), m.values("v", range(n), n * page - 3), dim ** -0.5,
                          True, 0, out, many=many)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), float((err / tol).max())


# ---- copies, and all of it together --------------------------------------------

@pytest.mark.parametrize("pairs,heads,dim,page", [(1, 1, 64, 64), (7, 3, 128, 64), (449, 1, 64, 64), (1000, 2, 64, 64),
                                                  (3, 5, 256, 256)])
def test_copies(pairs, heads, dim, page):
    import moe_decode_amd as md
    import torch
    rng = np.random.default_rng(pairs)
    n = 2 * pairs + 3
    m = Cache(n, heads, page, dim, rng)
    c = _to_gpu(m)
    order = rng.permutation(n)
    src, dst = order[:pairs].copy(), order[pairs:2 * pairs]
    src[pairs // 2] = src[0]            # one page copied twice
    md.kv_copy_pages(c, src.tolist(), dst.tolist())
    for name in "kv":
        m.c[name][dst], m.s[name][dst] = m.c[name][src], m.s[name][src]
    g = Cache(n, heads, page, dim, rng)
    _from_gpu(c, g)
    for name in "kv":
        assert np.array_equal(g.c[name], m.c[name]) and np.array_equal(g.s[name], m.s[name])
    with pytest.raises(md.MDError) as e:
        md.kv_copy_pages(c, [0], [n])
    assert e.value.name == "MD_ERR_INVALID_ARG"
    with pytest.raises(ValueError):
        md.kv_copy_pages(c, [0, 1], [2])


def test_refused_tensors():
    import moe_decode_amd as md
    import torch
    c = md.KVCache.empty(2, 2, 64)
    b = _batch([1], [1], [[0]])
    k = torch.zeros(1, 2, 64, device="cuda")
    with pytest.raises(ValueError):
        md.KVCache(c.k, c.k.transpose(2, 3), c.k_scale, c.v_scale)
    with pytest.raises(ValueError):
        md.KVCache(c.k, c.v, c.k_scale.double(), c.v_scale)
    for bad in (k[:, :1], torch.zeros(1, 2, 128, device="cuda")[:, :, ::2], k.cpu(), torch.zeros(2, 64, device="cuda")):
        with pytest.raises(ValueError):
            md.kv_append(c, b, bad, k)
    with pytest.raises(ValueError):
        md.kv_append(c, b, k, k.bfloat16())
    with pytest.raises((TypeError, ValueError)):
        md.kv_append(c, b, k.half(), k.half())
    with pytest.raises(md.MDError) as e:
        md.kv_attention(c, b, torch.zeros(1, 3, 64, device="cuda"))
    assert e.value.name == "MD_ERR_SHAPE"
    with pytest.raises(ValueError):
        md.kv_attention(c, b, torch.zeros(1, 4, 32, device="cuda"))
    with pytest.raises(ValueError):
        md.kv_attention(c, b, torch.zeros(1, 4, 64, device="cuda"), out=torch.zeros(2, 4, 64, device="cuda"))
    assert md.kv_attention(c, _batch([0], [0], [[0]]), torch.zeros(0, 4, 64, device="cuda")).shape == (0, 4, 64)


class _Layer:
    """An attention block in 8 bits and the c0 MoE layer behind it, each with
    its residual: hidden 256, 4 query heads on 2 key heads of 64."""

    def __init__(self, seed):
        import moe_decode_amd as md
        import torch
        from .gpu_common import moe_layer
        rng = np.random.default_rng(seed)

        def mat(n, k):
            return md.DevQMatrix("i8_row", n, k, torch.from_numpy(rng.integers(-127, 128, (n, k)).astype(np.int8)).cuda().view(-1),
                                 torch.from_numpy(rng.uniform(5e-4, 1e-3, n).astype(np.float32)).cuda())
        self.qkv, self.o, self.moe = mat(512, 256), mat(256, 256), moe_layer("c0")
        self.cache = md.KVCache.empty(12, 2, 64, 64)

    def __call__(self, x, batch, keep=None):
        import moe_decode_amd as md
        n = x.shape[0]
        qkv = md.i8_linear(self.qkv, x).view(n, 8, 64)
        md.kv_append(self.cache, batch, qkv[:, 4:6], qkv[:, 6:])
        a = md.kv_attention(self.cache, batch, qkv[:, :4])
        if keep is not None:
            keep.extend([qkv, a])
        h = md.add(x, md.i8_linear(self.o, a.view(n, 256)))
        return md.moe_layer_forward(self.moe, h, residual=h)


def test_a_decoder_layer_eager_captured_forked_and_compacted():
    """Two prompts, decode steps (captured; replayed with eager calls between),
    a fork that shares pages and then writes its own, rejected tokens given
    back, a compaction: every attention output against the definition on the
    cache's content, replays equal to eager calls on an equal cache."""
    import moe_decode_amd as md
    import torch
    L, E = _Layer(1), _Layer(1)
    kv = md.KVPages(12, 64, 3, 4)
    g = torch.Generator(device="cuda").manual_seed(7)

    def copies(pairs):
        for layer in (L, E):
            md.kv_copy_pages(layer.cache, [a for a, _ in pairs], [b for _, b in pairs])

    def batch(nq, seqs, max_q=None):
        return _batch(nq, [int(kv.lens[s]) for s in seqs], kv.tables[seqs], max_q, max_kv=256)

    def check(layer, b, nq, seqs, keep):
        m = Cache(12, 2, 64, 64, np.random.default_rng(0))
        _from_gpu(layer.cache, m)
        qkv, a = (t.cpu().numpy() for t in keep)
        at = 0
        for n, s in zip(nq, seqs):
            t = int(kv.lens[s])
            want, tol = attention(qkv[at:at + n, :4], m.values("k", kv.tables[s], t), m.values("v", kv.tables[s], t),
                                  0.125, True, 0, "f32", many=b.max_q * 2 > 64)
            assert (np.abs(a[at:at + n] - want) <= tol).all()
            at += n
    nq = [70, 33]
    for s, n in enumerate(nq):
        copies(kv.extend(s, n))
    x = torch.randn(103, 256, generator=g, device="cuda")
    keep = []
    b = batch(nq, [0, 1])
    y = L(x, b, keep)
    check(L, b, nq, [0, 1], keep)
    assert torch.equal(E(x, b), y)
    # decode: one graph, its batch's arrays rewritten between replays
    live = md.KVBatch(_i32([0, 1, 2]), _i32([1, 1]), _i32(np.zeros((2, 4))), 1, 256)
    xin = torch.zeros(2, 256, device="cuda")
    for s in (0, 1):
        copies(kv.extend(s, 1))
    live.kv_len.copy_(_i32(kv.lens[:2]))
    live.table.copy_(_i32(kv.tables[:2]))
    xin.copy_(torch.randn(2, 256, generator=g, device="cuda"))
    before = [t.clone() for t in (L.cache.k, L.cache.v, L.cache.k_scale, L.cache.v_scale)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        L(xin, live)                    # warms the allocator up
    torch.cuda.current_stream().wait_stream(st)
    for t, w in zip((L.cache.k, L.cache.v, L.cache.k_scale, L.cache.v_scale), before):
        t.copy_(w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yg = L(xin, live)
    for step in range(5):
        if step:
            for s in (0, 1):
                copies(kv.extend(s, 1))
            live.kv_len.copy_(_i32(kv.lens[:2]))
            live.table.copy_(_i32(kv.tables[:2]))
            xin.copy_(torch.randn(2, 256, generator=g, device="cuda"))
        graph.replay()
        keep = []
        ye = E(xin, live, keep)
        assert torch.equal(yg, ye), step
        check(E, live, [1, 1], [0, 1], keep)
        torch.cuda.synchronize()
    assert torch.equal(L.cache.k[kv.tables[0, 0]], E.cache.k[kv.tables[0, 0]])
    # a fork of the first sequence: shared pages, then a page of its own
    kv.fork(0, 2)
    pairs = kv.extend(2, 3)
    assert len(pairs) == 1
    copies(pairs)
    old = E.cache.k[pairs[0][0]].clone()
    keep, b = [], batch([3], [2], max_q=3)
    x3 = torch.randn(3, 256, generator=g, device="cuda")
    E(x3, b, keep)
    check(E, b, [3], [2], keep)
    assert torch.equal(E.cache.k[pairs[0][0]], old)
    # two of them rejected, another token instead; then the second sequence goes and the rest moves together
    kv.truncate(2, int(kv.lens[2]) - 2)
    copies(kv.extend(2, 1))
    keep, b = [], batch([1], [2])
    E(x3[:1].contiguous(), b, keep)
    check(E, b, [1], [2], keep)
    kv.truncate(1)
    b = batch([1], [2])
    q = torch.randn(1, 4, 64, generator=g, device="cuda")
    want = md.kv_attention(E.cache, b, q)
    pairs = kv.compact()
    assert pairs
    copies(pairs)
    assert torch.equal(md.kv_attention(E.cache, batch([1], [2]), q), want)


def test_two_streams_at_once():
    """Two calls in flight, each with its own workspace."""
    import moe_decode_amd as md
    import torch
    Hkv, dim, page, L = 2, 128, 64, 20000
    rng = np.random.default_rng(2)
    table, n = _tables([L], page, rng)
    c = _to_gpu(Cache(n, Hkv, page, dim, rng))
    b = _batch([1], [L], table)
    qs = [_rn(rng, (1, 8, dim), "f32")[0] for _ in range(2)]
    want = [md.kv_attention(c, b, q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for q, st in zip(qs, streams):
            with torch.cuda.stream(st):
                got.append(md.kv_attention(c, b, q))
        torch.cuda.synchronize()
        assert all(torch.equal(a, w) for a, w in zip(got, want))


def test_a_captured_call_follows_the_lengths():
    """One graph of append and attention over long contexts, its batch's arrays
    and pages rewritten between the replays; every replay equals the eager call
    (long and short sequences, one without rows)."""
    import moe_decode_amd as md
    import torch
    Hkv, G, dim, page = 2, 4, 128, 64
    rng = np.random.default_rng(21)
    cases = [([1, 1, 1], [1900, 3, 700]), ([1, 0, 2], [64, 500, 2000]), ([2, 1, 0], [129, 4999, 0])]
    tables = [_tables(l, page, rng) for _, l in cases]
    n = max(t[1] for t in tables)
    m = Cache(n, Hkv, page, dim, rng)
    live, ref = _to_gpu(m), _to_gpu(m)
    rows = 3
    b = md.KVBatch(_i32([0, 0, 0, 0]), _i32([0, 0, 0]), _i32(np.zeros((3, 80))), 2, 5000)
    q, k, v = (torch.zeros(rows, h, dim, device="cuda") for h in (Hkv * G, Hkv, Hkv))
    out = torch.empty(rows, Hkv * G, dim, device="cuda")
    ws = torch.empty(md.kv_attention_workspace_size(live, b, rows, Hkv * G), dtype=torch.uint8, device="cuda")

    def call(c, o, w=None):
        md.kv_append(c, b, k, v)
        md.kv_attention(c, b, q, out=o, workspace=w)
    call(live, out, ws)                     # (no rows: writes nothing)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(live, out, ws)
    for turn in range(6):
        (nq, lens), (table, _) = cases[turn % 3], tables[turn % 3]
        b.q_start.copy_(_i32(np.concatenate([[0], np.cumsum(nq)])))
        b.kv_len.copy_(_i32(lens))
        b.table.zero_()
        b.table[:, :table.shape[1]].copy_(_i32(np.maximum(table, 0)))
        for t in (q, k, v):
            t.copy_(torch.from_numpy(rng.standard_normal(t.shape).astype(np.float32)))
        g.replay()
        want = torch.empty_like(out)
        call(ref, want)
        r = sum(nq)
        assert torch.equal(out[:r], want[:r]), turn
        assert torch.equal(live.k, ref.k) and torch.equal(live.v, ref.v) and torch.equal(live.k_scale, ref.k_scale)
        torch.cuda.synchronize()
