"""Attention over trees of drafts and over windows with sinks on the GPU, within
the bound derived in kv_model.py of the definition in 64 bits on the codes the
cache holds; the trees' masks and positions; and a step that checks drafts, made
of all the operators around it, eager and captured."""
import numpy as np
import pytest

from . import step_model as M
from .gpu_common import require_gpu
from .kv_model import Cache, many_columns
from .test_gpu_kv import _batch, _dt, _i32, _rn, _tables, _to_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _tree(rng, n, kind):
    if kind == "chain":
        return list(range(-1, n - 1))
    if kind == "roots":
        return [-1] * n
    return [-1] * min(n, 1) + [int(rng.integers(max(-1, i - 7), i)) for i in range(1, n)]


def _run(seqs, Hkv, G, dim, page, xt, yt, kind=None, window=0, sinks=0, seed=0, words=0, holes=False):
    """seqs: (new, length) of each; kind: the trees', or None for positions alone."""
    import moe_decode_amd as md
    import torch
    rng = np.random.default_rng(seed)
    nq, lens = [a for a, _ in seqs], [b for _, b in seqs]
    table, n_pages = _tables(lens, page, rng, spare=1)
    m = Cache(n_pages, Hkv, page, dim, rng)
    c, b = _to_gpu(m), _batch(nq, lens, table)
    q, qn = _rn(rng, (sum(nq), G * Hkv, dim), xt)
    bits, masks = [None] * sum(nq), None
    if kind:
        bits = [x for n in nq for x in M.tree_bits(_tree(rng, n, kind))]
        if holes:       # rows that see nothing of the run, not even themselves
            bits = [[] if i % 3 == 1 else x for i, x in enumerate(bits)]
        w = max(words, -(-max(nq) // 64))
        masks = M.pack(bits, w)
        at = 0
        for n in nq:    # bits past the run mean nothing
            past = [list(range(n, 64 * w)) for _ in range(n)]
            masks[at:at + n] |= M.pack(past, w)
            at += n
        masks = torch.from_numpy(masks).cuda()
    out = md.kv_attention(c, b, q, window=window, sinks=sinks, tree=masks, out_dtype=_dt(yt)).float().cpu().numpy()
    many, at = many_columns(max(nq), G, dim, yt), 0
    for s, (n, length) in enumerate(seqs):
        if not n:
            continue
        k, v = m.values("k", table[s], length), m.values("v", table[s], length)
        seen = [M.visible(length, n, i, window if window < max(lens) else 0, sinks, bits[at + i]) for i in range(n)]
        o, tol = M.attend(qn[at:at + n], k, v, dim ** -0.5, seen, yt, many)
        err = np.abs(out[at:at + n] - o)
        assert (err <= tol).all(), (s, np.argwhere(err > tol)[:4].tolist(), float((err / tol).max()))
        at += n


TREES = [   # (new, length) of each sequence, key heads, queries each, channels, page
    ([(1, 1)], 1, 1, 64, 64),
    ([(5, 5), (1, 64), (3, 3)], 2, 4, 128, 64),
    ([(12, 300), (7, 65), (0, 10), (1, 129)], 2, 8, 256, 128),
    ([(33, 33), (64, 64), (20, 84), (17, 4000)], 1, 2, 64, 64),
    ([(65, 140), (63, 700)], 2, 1, 128, 64),                     # a run of two words
    ([(30, 3000), (9, 2100)], 4, 4, 128, 256),                   # many columns
    ([(200, 260), (130, 1000)], 1, 4, 64, 64),
    ([(40, 900)], 1, 16, 256, 64),
    ([(61, 9000)], 1, 2, 64, 128),
]


@pytest.mark.parametrize("case", range(len(TREES)))
@pytest.mark.parametrize("xt,yt", [("f32", "f32"), ("bf16", "bf16")])
def test_trees(case, xt, yt):
    seqs, Hkv, G, dim, page = TREES[case]
    _run(seqs, Hkv, G, dim, page, xt, yt, "tree", seed=case)
    _run(seqs, Hkv, G, dim, page, xt, yt, "roots", seed=case, words=5, holes=True)


@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 2), (64, 64), (100, 5), (130, 200), (1000, 1), (5000, 3)])
@pytest.mark.parametrize("xt,yt", [("f32", "f32"), ("bf16", "bf16")])
def test_trees_in_a_window(window, sinks, xt, yt):
    _run([(12, 300), (7, 65), (1, 1500)], 2, 4, 64, 64, xt, yt, "tree", window, sinks, seed=window)
    _run([(70, 700), (5, 5)], 1, 2, 128, 128, xt, yt, "tree", window, sinks, seed=window, holes=True)


SINKS = [
    ([(1, 1), (1, 64), (1, 65), (1, 2000)], 2, 4, 128, 64),
    ([(1, 20000), (1, 15000)], 1, 8, 64, 128),                   # dealt out and joined
    ([(3, 700), (16, 16), (0, 9), (9, 1000)], 2, 2, 256, 64),
    ([(300, 1000), (257, 257)], 1, 4, 128, 64),                  # many columns
    ([(900, 1800)], 1, 1, 64, 256),
    ([(1, 5000)] * 3, 8, 1, 64, 64),
]


@pytest.mark.parametrize("case", range(len(SINKS)))
@pytest.mark.parametrize("window,sinks", [(1, 1), (64, 4), (65, 64), (200, 129), (1000, 700), (7, 100000)])
@pytest.mark.parametrize("xt,yt", [("f32", "f32"), ("bf16", "bf16")])
def test_sinks(case, window, sinks, xt, yt):
    seqs, Hkv, G, dim, page = SINKS[case]
    _run(seqs, Hkv, G, dim, page, xt, yt, None, window, sinks, seed=case)


@pytest.mark.parametrize("nq,lens,G,dim", [([5, 64], [70, 300], 2, 64), ([33, 1], [2000, 1], 8, 128), ([9], [9], 4, 256)])
def test_chains_are_causal_and_open_masks_change_nothing(nq, lens, G, dim):
    """A tree without branches gives the bits of plain causal attention, and so do
    sinks without a window, a window past every position, and a zero window.  (fp32
    outputs of many columns of 128 channels or more take a tree's scores in other
    blocks: both calls then round each weight by 2^-23 and sum up to L of them, each
    sum off by L u of its terms' sizes, numerator and denominator: 2 (2 L u + 2^-22)
    max |v| apart at most.)"""
    import moe_decode_amd as md
    import torch
    rng = np.random.default_rng(dim)
    table, n = _tables(lens, 64, rng)
    c = _to_gpu(Cache(n, 2, 64, dim, rng))
    b = _batch(nq, lens, table)
    q, _ = _rn(rng, (sum(nq), 2 * G, dim), "f32")
    parents = _i32([p for a in nq for p in range(-1, a - 1)])
    masks, pos = md.kv_tree(b, parents)
    assert pos.tolist() == [l - a + i for a, l in zip(nq, lens) for i in range(a)]
    for dt in (torch.float32, torch.bfloat16):
        want = md.kv_attention(c, b, q, out_dtype=dt)
        got = md.kv_attention(c, b, q, tree=masks, out_dtype=dt)
        if dt == torch.float32 and dim > 64 and many_columns(max(nq), G, dim, "f32"):
            most = 127 * c.v_scale.max().item()
            assert (got - want).abs().max() <= 2 * (2 * max(lens) * M.U + 2.0 ** -22) * most
        else:
            assert torch.equal(got, want)
        assert torch.equal(md.kv_attention(c, b, q, sinks=5, out_dtype=dt), want)
        assert torch.equal(md.kv_attention(c, b, q, window=max(lens), sinks=5, tree=masks, out_dtype=dt), got)
        # sinks that reach up to the window leave nothing out
        got = md.kv_attention(c, b, q, window=3, sinks=max(lens), out_dtype=dt)
        assert (got.float() - want.float()).abs().max() <= 2.0 ** (-7 if dt == torch.bfloat16 else -12)


def test_what_a_row_does_not_see_does_not_reach_it():
    """A page whose scale is none, and a page number that is none: NaN only in the
    rows that see one of their tokens."""
    import moe_decode_amd as md
    rng = np.random.default_rng(8)
    table = np.array([[3, 1, 4, 0, 2]], np.int32)
    m = Cache(5, 2, 64, 64, rng)
    c = _to_gpu(m)
    b = _batch([3], [300], table)
    q, _ = _rn(rng, (3, 4, 64), "f32")
    masks = _tree_masks([[0], [0, 1], [2]])
    good = md.kv_attention(c, b, q, window=90, sinks=10, tree=masks)
    c.k_scale[1] = float("nan")         # positions 64..127: outside the window of all, and no sinks
    assert (md.kv_attention(c, b, q, window=90, sinks=10, tree=masks) == good).all()
    got = md.kv_attention(c, b, q, window=90, sinks=70, tree=masks)
    assert got.isnan().all()
    b2 = _batch([3], [300], np.array([[3, 99, 4, 0, 2]], np.int32))
    assert (md.kv_attention(c, b2, q, window=90, sinks=10, tree=masks) == good).all()
    assert md.kv_attention(c, b2, q, tree=masks).isnan().all()
    c.k_scale[2] = float("nan")         # the page with the run's tokens: all see one of them, unless they see none
    none = _tree_masks([[0], [], [2]])
    got = md.kv_attention(c, _batch([3], [259], table), q, window=40, sinks=0, tree=none)
    assert got[0].isnan().all() and got[2].isnan().all() and not got[1].isnan().any()


def _tree_masks(bits):
    import torch
    return torch.from_numpy(M.pack(bits, 1)).cuda()


def test_bad_sequences_and_rows_behind():
    import moe_decode_amd as md
    import torch
    rng = np.random.default_rng(9)
    c = _to_gpu(Cache(4, 1, 64, 64, rng))
    table = np.zeros((3, 2), np.int32)
    b = _batch([2, 2, 2], [100, 129, 3], table, max_q=2, max_kv=128)      # the second is longer than it may be
    q, _ = _rn(rng, (8, 2, 64), "f32")
    out = torch.full((8, 2, 64), 7.0, device="cuda")
    masks = torch.from_numpy(M.pack([[0], [1]] * 4, 1)).cuda()
    md.kv_attention(c, b, q, tree=masks, out=out)
    assert out[2:4].isnan().all() and not out[:2].isnan().any() and not out[4:6].isnan().any() and (out[6:] == 7.0).all()
    # a run longer than its sequence: the tokens before position 0 are none
    short = _batch([3], [1], np.zeros((1, 1), np.int32))
    got = md.kv_attention(c, short, q[:3], tree=torch.from_numpy(M.pack([[0], [0, 1], [0, 1, 2]], 1)).cuda())
    assert (got[:2] == 0).all() and not (got[2] == 0).all()


@pytest.mark.parametrize("yt", ["f32", "bf16"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (900, 70)])
def test_captured_calls_follow_lengths_and_trees(yt, window, sinks):
    """Many columns whose splits are dealt out by the lengths on the device: a graph
    replayed over other lengths (from nothing cached to the bound) and other trees."""
    import moe_decode_amd as md
    import torch
    rng = np.random.default_rng(21)
    nq, most = [40, 0, 33], 9000
    table, n = _tables([most] * 3, 64, rng)
    m = Cache(n, 1, 64, 64, rng)
    c, b = _to_gpu(m), _batch(nq, [most] * 3, table)
    q, qn = _rn(rng, (73, 4, 64), "bf16")
    masks, pos = md.kv_tree(b, _i32([p for a in nq for p in _tree(rng, a, "tree")]))
    kw = dict(window=window, sinks=sinks, tree=masks, out_dtype=_dt(yt))
    md.kv_attention(c, b, q, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = md.kv_attention(c, b, q, **kw)
    for lens in ([40, 0, 9000], [8999, 17, 33], [3000, 5, 2500], [9000, 9000, 9000]):
        bits = [x for a in nq for x in M.tree_bits(_tree(rng, a, "tree"))]
        masks.copy_(torch.from_numpy(M.pack(bits, 1)))
        b.kv_len.copy_(_i32(lens))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, md.kv_attention(c, b, q, **kw))
        at = 0
        for s, (a, length) in enumerate(zip(nq, lens)):
            if not a:
                continue
            rows = sorted({0, a // 2, a - 1})
            seen = [M.visible(length, a, i, window, sinks, bits[at + i]) for i in rows]
            o, tol = M.attend(qn[[at + i for i in rows]], m.values("k", table[s], length), m.values("v", table[s], length),
                              64 ** -0.5, seen, yt, True)
            err = np.abs(got[[at + i for i in rows]].float().cpu().numpy() - o)
            assert (err <= tol).all(), (lens, s, float((err / tol).max()))
            at += a


def test_calls_on_two_streams():
    """Two calls at once, each on its own stream and workspace."""
    import moe_decode_amd as md
    import torch
    rng = np.random.default_rng(22)
    table, n = _tables([5000, 3000], 64, rng)
    c = _to_gpu(Cache(n, 2, 64, 64, rng))
    b = _batch([64, 40], [5000, 3000], table)
    q = [_rn(rng, (104, 8, 64), "f32")[0] for _ in range(2)]
    masks, _ = md.kv_tree(b, _i32([p for a in (64, 40) for p in _tree(rng, a, "tree")]))
    x = torch.randn(2100, 4096, device="cuda")
    W = torch.randn(256, 4096, device="cuda") * 0.02
    r = md.Routing(8, "sigmoid")
    want = [md.kv_attention(c, b, t, tree=masks) for t in q] + list(md.moe_route(x, W, r))
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(5):
        got = [md.kv_attention(c, b, t, tree=masks, stream=st) for t, st in zip(q, s)] + \
            list(md.moe_route(x, W, r, stream=s[2]))
        torch.cuda.synchronize()
        assert all(torch.equal(a, w) for a, w in zip(got, want))


@pytest.mark.parametrize("nq", [[1], [5, 0, 64], [65, 1, 130], [1024]])
def test_masks_and_positions(nq):
    import moe_decode_amd as md
    import torch
    rng = np.random.default_rng(sum(nq))
    lens = [n + int(rng.integers(0, 500)) for n in nq]
    parents, bits, pos = [], [], []
    for n, l in zip(nq, lens):
        p = _tree(rng, n, "tree") if n else []
        if n > 20:
            p[11], p[12], p[17], p[18] = 12, 12, -2, 17       # not before itself, itself, none; a child of one
        for i, x in enumerate(M.tree_bits(p)):
            bits.append(x)
            pos.append(-1 if x is None else l - n + len(x) - 1)
        parents += p
    b = _batch(nq, lens, np.zeros((len(nq), 30), np.int32))
    masks, got = md.kv_tree(b, _i32(parents))
    assert np.array_equal(masks.cpu().numpy(), M.pack(bits, masks.shape[1]))
    assert got.tolist() == pos
    wide = torch.full((len(parents) + 1, masks.shape[1] + 2), -1, dtype=torch.int64, device="cuda")
    md.kv_tree(b, _i32(parents), masks=wide[:-1])
    assert np.array_equal(wide[:-1].cpu().numpy(), M.pack(bits, wide.shape[1])) and (wide[-1] == -1).all()


# ---- a step that checks drafts ---------------------------------------------

class _Step:
    """One layer and a head: projection, norms and rotation, append, attention over
    the tree, output projection, experts by balanced groups, logits, log
    probabilities of each token's drafts."""

    H, Hq, Hkv, D, E, k, V = 2048, 16, 4, 128, 128, 8, 3001

    def __init__(self):
        import moe_decode_amd as md
        import torch

        from .gpu_common import moe_layer
        g = torch.Generator(device="cuda").manual_seed(11)

        def matrix(n, c):
            return md.DevQMatrix("i8_row", n, c, torch.randint(-127, 128, (n * c,), generator=g, device="cuda",
                                                               dtype=torch.int8),
                                 torch.full((n,), 0.6 / 73 / c ** 0.5, device="cuda"))
        self.qkv = matrix((self.Hq + 2 * self.Hkv) * self.D, self.H)
        self.o, self.head = matrix(self.H, self.Hq * self.D), matrix(self.V, self.H)
        self.layer = moe_layer("c3")
        self.routing = md.Routing(self.k, "sigmoid", 0.05 * torch.randn(self.E, generator=g, device="cuda"), 8, 4, True,
                                  scale=2.5)
        self.w = [1 + 0.1 * torch.randn(self.D, generator=g, device="cuda") for _ in range(2)]
        self.inv = (10000.0 ** (-torch.arange(0, self.D, 2) / self.D)).cuda()

    def __call__(self, cache, batch, x, parents, tokens):
        import moe_decode_amd as md
        n = x.shape[0]
        masks, pos = md.kv_tree(batch, parents)
        qkv = md.i8_linear(self.qkv, x).view(n, -1, self.D)
        q, k, v = qkv[:, :self.Hq], qkv[:, self.Hq:self.Hq + self.Hkv], qkv[:, self.Hq + self.Hkv:]
        q, k = md.qk_norm_rope(q, k, pos, self.inv, *self.w, q_out=q, k_out=k)
        md.kv_append(cache, batch, k, v)
        a = md.kv_attention(cache, batch, q, tree=masks)
        h = md.add(x, md.i8_linear(self.o, a.view(n, -1)))
        y = md.add(h, md.moe_layer_forward(self.layer, h, routing=self.routing))
        logits = md.i8_linear(self.head, y)
        return dict(pos=pos, q=q, k=k, a=a, h=h, y=y, logits=logits, lp=md.token_logprobs(logits, tokens, top=4))


def test_a_step_over_drafts_eager_and_captured():
    """Each operator's output against its model on its own input; the same step
    captured and replayed over other trees and lengths."""
    import moe_decode_amd as md
    import torch
    rng = np.random.default_rng(12)
    step = _Step()
    nq, lens = [9, 5], [9 + 170, 5 + 60]
    pages = md.KVPages(16, 64, 2, 4)
    for s, l in enumerate(lens):
        pages.extend(s, l)
    m = Cache(16, step.Hkv, 64, step.D, rng)
    cache = _to_gpu(m)
    b = _batch(nq, lens, pages.tables, max_kv=256)
    x = torch.randn(14, step.H, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    trees = [_tree(rng, n, "tree") for n in nq]
    parents, tokens = _i32(sum(trees, [])), _i32(rng.integers(0, step.V, (14, 3)))
    r = step(cache, b, x, parents, tokens)
    bits = [t for p in trees for t in M.tree_bits(p)]
    pos = [l - n + len(t) - 1 for n, l, p in zip(nq, lens, trees) for t in M.tree_bits(p)]
    assert r["pos"].tolist() == pos
    q = r["q"].cpu().numpy()
    from .test_gpu_kv import _from_gpu
    _from_gpu(cache, m)
    at = 0
    for s, (n, l) in enumerate(zip(nq, lens)):
        kk, vv = m.values("k", pages.tables[s], l), m.values("v", pages.tables[s], l)
        o, tol = M.attend(q[at:at + n], kk, vv, step.D ** -0.5, [M.visible(l, n, i, 0, 0, bits[at + i]) for i in range(n)],
                          "f32", many_columns(max(nq), 4, step.D, "f32"))
        assert (np.abs(r["a"][at:at + n].cpu().numpy() - o) <= tol).all()
        # the keys that the cache holds are the rotated ones, within a step of their page
        step_size = m.s["k"][pages.tables[s]][[p // 64 for p in range(l - n, l)]]
        assert (np.abs(kk[l - n:] - r["k"][at:at + n].cpu().numpy()) <= 0.51 * step_size[:, :, None]).all()
        at += n
    i, g = md.moe_route(r["h"], step.layer.Wr, step.routing, bias=step.layer.bias)
    assert torch.equal(r["y"], md.add(r["h"], md.moe_experts_forward(step.layer, r["h"], i, g)))
    # (the layer's random experts leave log probabilities near -2e4, whose rounding alone is 2^-24 2e4 = 1.2e-3)
    lp, tol, _, _ = M.logprobs(r["logits"].cpu().numpy(), 1.0)
    rows, at = np.arange(14)[:, None], tokens.cpu().numpy()
    assert (np.abs(r["lp"].logprobs.cpu().numpy() - lp[rows, at]) <= tol[rows, at]).all()
    # the accepted tokens stay, the others' pages go back
    pages.truncate(0, 170 + 2)
    pages.truncate(1, 60)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(cache, b, x, parents, tokens)
    for i in range(3):
        x.copy_(torch.randn(14, step.H, device="cuda"))
        parents.copy_(_i32(sum((_tree(rng, n, "tree") for n in nq), [])))
        b.kv_len.copy_(_i32([100 + 30 * i, 40 + i]))
        keep = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
        graph.replay()
        torch.cuda.synchronize()
        mine = {k: (v if k == "lp" else v.clone()) for k, v in got.items()}
        lp = [t.clone() for t in got["lp"]]
        for t, was in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), keep):
            t.copy_(was)
        want = step(cache, b, x, parents, tokens)
        for name in ("pos", "q", "k", "a", "h", "y", "logits"):
            assert torch.equal(mine[name], want[name]), (i, name)
        assert all(torch.equal(p, w) for p, w in zip(lp, want["lp"]))
