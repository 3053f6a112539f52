"""Trees of drafts beside a sliding window that is shorter than their paths, on the
GPU: with masks made for the window a row sees the tokens that its path gives when
they are decoded one by one, a chain those of a causal run."""
import numpy as np
import pytest

from . import step_model as M
from .gpu_common import require_gpu
from .kv_model import Cache, many_columns
from .test_gpu_kv import _batch, _dt, _i32, _rn, _tables, _to_gpu
from .test_gpu_kv_tree import _tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _kept(path, base, window, sinks):
    """Of a token's path (numbers within the run, the root first): those that the
    window or the first positions leave."""
    p = base + len(path) - 1
    return [j for k, j in enumerate(path) if not window or base + k > p - window or base + k < sinks]


def _seen(path, base, window, sinks):
    """The cache slots that it sees: its place in the text decides, before the run
    and on its path."""
    p = base + len(path) - 1
    before = [c for c in range(base) if not window or c > p - window or c < sinks]
    return np.array(before + sorted(base + j for j in _kept(path, base, window, sinks)), np.int64)


SHAPES = [   # (new, length) of each sequence, key heads, queries each, channels, page
    ([(12, 300), (7, 7), (1, 1500), (9, 11)], 2, 4, 64, 64),
    ([(70, 700), (5, 5), (0, 30), (130, 131)], 1, 2, 128, 128),
    ([(40, 900), (64, 70)], 1, 4, 256, 64),
    ([(33, 4000)], 2, 8, 128, 64),                               # many columns, splits
    ([(61, 9000)], 1, 2, 64, 128),                               # dealt out
]


@pytest.mark.parametrize("kind", ["chain", "tree"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 2), (8, 0), (20, 40), (64, 3), (5, 1000)])
@pytest.mark.parametrize("case", range(len(SHAPES)))
@pytest.mark.parametrize("yt", ["f32", "bf16"])
def test_paths_longer_than_the_window(case, window, sinks, kind, yt):
    import moe_decode_amd as md
    seqs, Hkv, G, dim, page = SHAPES[case]
    rng = np.random.default_rng(100 * case + window)
    nq, lens = [a for a, _ in seqs], [b for _, b in seqs]
    table, n_pages = _tables(lens, page, rng, spare=1)
    m = Cache(n_pages, Hkv, page, dim, rng)
    c, b = _to_gpu(m), _batch(nq, lens, table)
    q, qn = _rn(rng, (sum(nq), G * Hkv, dim), yt)
    trees = [_tree(rng, n, kind) for n in nq]
    paths = [M.tree_bits(t) for t in trees]
    masks, pos = md.kv_tree(b, _i32(sum(trees, [])), window=window, sinks=sinks)
    kept = [_kept(p, l - n, window, sinks) for n, l, ps in zip(nq, lens, paths) for p in ps]
    assert np.array_equal(masks.cpu().numpy(), M.pack(kept, masks.shape[1]))
    assert pos.tolist() == [l - n + len(p) - 1 for n, l, ps in zip(nq, lens, paths) for p in ps]
    kw = dict(window=window, sinks=sinks, out_dtype=_dt(yt))
    out = md.kv_attention(c, b, q, tree=masks, **kw).float().cpu().numpy()
    causal = md.kv_attention(c, b, q, **kw).float().cpu().numpy()
    many, at = many_columns(max(nq), G, dim, yt), 0
    for s, (n, length) in enumerate(seqs):
        if not n:
            continue
        k, v = m.values("k", table[s], length), m.values("v", table[s], length)
        rows = sorted({0, 1, n // 3, n // 2, n - 2, n - 1} & set(range(n)))
        seen = [_seen(paths[s][i], length - n, window, sinks) for i in rows]
        if kind == "chain":
            assert all(np.array_equal(a, M.visible(length, n, i, window, sinks)) for a, i in zip(seen, rows))
        at_rows = [at + i for i in rows]
        o, tol = M.attend(qn[at_rows], k, v, dim ** -0.5, seen, yt, many)
        for got in [out, causal] if kind == "chain" else [out]:
            err = np.abs(got[at_rows] - o)
            assert (err <= tol).all(), (s, np.argwhere(err > tol)[:4].tolist(), float((err / tol).max()))
        at += n


def test_no_window_keeps_every_ancestor_and_bad_chains_have_none():
    import moe_decode_amd as md
    import torch
    rng = np.random.default_rng(3)
    parents = _tree(rng, 100, "tree")
    parents[30], parents[31] = 30, 30        # not before itself; a child of one
    b = _batch([100], [140], np.zeros((1, 3), np.int32))
    masks, pos = md.kv_tree(b, _i32(parents))
    assert np.array_equal(masks.cpu().numpy(), M.pack(M.tree_bits(parents), 2))
    wide, wpos = md.kv_tree(b, _i32(parents), window=1000, sinks=5)
    assert torch.equal(wide, masks) and torch.equal(wpos, pos)
    few, fpos = md.kv_tree(b, _i32(parents), window=2)
    assert torch.equal(fpos, pos) and (few[30] == 0).all() and (few[31] == 0).all() and pos[31] == -1
    keep = [None if p is None else _kept(p, 40, 2, 0) for p in M.tree_bits(parents)]
    assert np.array_equal(few.cpu().numpy(), M.pack(keep, 2))


@pytest.mark.parametrize("sinks", [0, 1])
def test_places_before_the_text_are_no_first_positions(sinks):
    """A run longer than its sequence: its first tokens stand at -2 and -1, and no sinks hold them."""
    import moe_decode_amd as md
    b = _batch([3], [1], np.zeros((1, 1), np.int32))
    masks, pos = md.kv_tree(b, _i32([-1, 0, 1]), window=1, sinks=sinks)
    assert pos.tolist() == [-2, -1, 0]
    assert np.array_equal(masks.cpu().numpy(), M.pack([[0], [1], [2]], 1))
