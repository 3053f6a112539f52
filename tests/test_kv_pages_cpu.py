"""The cache's page bookkeeping (host code) against a model that keeps each
table as a list and looks for free pages by set difference."""
import numpy as np
import pytest

import moe_decode_amd as md

from .kv_model import Pages


def _same(kv, m, seqs):
    for s in seqs:
        t = m.tables.get(s, [])
        assert kv.tables[s, :len(t)].tolist() == t, s
    assert kv.n_free == m.n - len(m.used())
    assert kv.refs.tolist() == [m.refs(p) for p in range(m.n)]


@pytest.mark.parametrize("seed", range(4))
def test_random_runs_match_the_model(seed):
    rng = np.random.default_rng(seed)
    n, page, S, cap = 40, 64, 6, 12
    kv, m = md.KVPages(n, page, S, cap), Pages(n, page)
    lens = [0] * S
    m.tables = {s: [] for s in range(S)}
    content = {}        # page -> what its copies and writers have made of it: a list of (sequence, position) marks
    seen = {s: [] for s in range(S)}
    refused = 0
    for _ in range(600):
        op, s = rng.choice(["extend", "extend", "fork", "truncate", "compact"]), int(rng.integers(S))
        if op == "extend":
            k = int(rng.integers(0, 150))
            t, have, want = m.tables[s], -(-lens[s] // page), -(-(lens[s] + k) // page)
            copy = k > 0 and lens[s] % page and m.refs(t[have - 1]) > 1
            if want > cap or want - have + bool(copy) > n - len(m.used()):
                with pytest.raises(md.MDError) as e:
                    kv.extend(s, k)
                assert e.value.name == ("MD_ERR_SHAPE" if want > cap else "MD_ERR_UNSUPPORTED")
                refused += 1
            else:
                pairs = kv.extend(s, k)
                if copy:
                    old, new = t[have - 1], m.take()
                    t[have - 1] = new
                    assert pairs == [(old, new)]
                    content[new] = list(content[old])
                else:
                    assert pairs == []
                for _ in range(want - have):
                    t.append(m.take())
                for pos in range(lens[s], lens[s] + k):
                    mark = int(rng.integers(1 << 30))
                    seen[s].append(mark)
                    c = content.setdefault(t[pos // page], [])
                    c[pos % page:] = [mark]
                lens[s] += k
        elif op == "fork":
            to = int(rng.integers(S))
            if to == s or lens[to]:
                with pytest.raises(ValueError):
                    kv.fork(s, to)
            else:
                k = int(rng.integers(0, lens[s] + 1))
                kv.fork(s, to, k)
                m.tables[to], lens[to], seen[to] = m.tables[s][: -(-k // page)], k, seen[s][:k]
                m.tables[to] = list(m.tables[to])
        elif op == "truncate":
            k = int(rng.integers(0, lens[s] + 1)) if rng.random() < 0.5 else 0
            kv.truncate(s, k)
            m.tables[s], lens[s], seen[s] = m.tables[s][: -(-k // page)], k, seen[s][:k]
        else:
            used = sorted(m.used())
            pairs = kv.compact()
            free = [p for p in range(len(used)) if p not in m.used()]
            want = list(zip([p for p in used if p >= len(used)], free))
            assert pairs == want
            to = dict(want)
            for p, q in want:
                content[q] = content.pop(p)
            m.tables = {k: [to.get(p, p) for p in t] for k, t in m.tables.items()}
            assert m.used() == set(range(len(used)))
        _same(kv, m, range(S))
        # what each sequence wrote is what its pages hold
        for q in range(S):
            assert [content[m.tables[q][p // page]][p % page] for p in range(lens[q])] == seen[q]
    assert refused      # the run reached full caches or tables


def _arrays(n):
    refs, free = np.zeros(n, np.int32), np.zeros(n, np.int32)
    st = md.KVPagesState(n, 64, refs.ctypes.data, free.ctypes.data, 0)
    return refs, free, st


def test_refusals_change_nothing():
    import ctypes
    L = md.lib()
    refs, free, st = _arrays(8)
    P = ctypes.byref
    assert md.STATUS[L.md_kv_pages_reset(None)] == "MD_ERR_INVALID_ARG"
    assert L.md_kv_pages_reset(P(st)) == 0 and st.n_free == 8
    a, b, k = (ctypes.c_int32 * 8)(), (ctypes.c_int32 * 8)(), ctypes.c_int32(7)
    t = np.full(8, -5, np.int32)
    tp = t.ctypes.data

    def name(rc):
        return md.STATUS[rc]
    assert L.md_kv_pages_extend(P(st), tp, 8, 0, 130, a, b, P(k)) == 0
    assert t.tolist() == [0, 1, 2, -5, -5, -5, -5, -5] and k.value == 0 and st.n_free == 5
    before = refs.copy()
    assert name(L.md_kv_pages_extend(P(st), tp, 8, 130, 129, a, b, P(k))) == "MD_ERR_SHAPE"
    assert name(L.md_kv_pages_extend(P(st), tp, 3, 130, 200, a, b, P(k))) == "MD_ERR_SHAPE"
    assert name(L.md_kv_pages_extend(P(st), tp, 99, 130, 64 * 9, a, b, P(k))) == "MD_ERR_UNSUPPORTED"
    assert name(L.md_kv_pages_extend(P(st), None, 8, 0, 1, a, b, P(k))) == "MD_ERR_INVALID_ARG"
    assert name(L.md_kv_pages_extend(P(st), tp, 8, 256, 300, a, b, P(k))) == "MD_ERR_INVALID_ARG"   # entry 3 names none
    u = np.array([0, 6], np.int32)                                                                  # 6 is free
    assert name(L.md_kv_pages_fork(P(st), u.ctypes.data, 100, tp, 8)) == "MD_ERR_INVALID_ARG"
    assert name(L.md_kv_pages_fork(P(st), tp, 100, u.ctypes.data, 1)) == "MD_ERR_SHAPE"
    assert name(L.md_kv_pages_truncate(P(st), tp, 10, 20)) == "MD_ERR_SHAPE"
    twice = np.array([0, 0], np.int32)
    assert name(L.md_kv_pages_truncate(P(st), twice.ctypes.data, 100, 0)) == "MD_ERR_INVALID_ARG"
    lens = np.array([64], np.int32)                                                                 # pages 1, 2 unnamed
    assert name(L.md_kv_pages_compact(P(st), tp, 8, lens.ctypes.data, 1, a, b, P(k))) == "MD_ERR_INVALID_ARG"
    lens[0] = 64 * 9
    assert name(L.md_kv_pages_compact(P(st), tp, 8, lens.ctypes.data, 1, a, b, P(k))) == "MD_ERR_SHAPE"
    assert name(L.md_kv_pages_compact(P(st), None, 8, lens.ctypes.data, 1, a, b, P(k))) == "MD_ERR_INVALID_ARG"
    assert refs.tolist() == before.tolist() and st.n_free == 5
    assert t.tolist() == [0, 1, 2, -5, -5, -5, -5, -5] and k.value == 0
    # the free pages still come lowest first
    lens[0] = 130
    assert L.md_kv_pages_extend(P(st), tp, 8, 130, 64 * 8, a, b, P(k)) == 0
    assert t.tolist() == list(range(8)) and st.n_free == 0


def test_lengths_of_zero_and_one():
    kv = md.KVPages(4, 128, 3, 4)
    assert kv.extend(0, 0) == [] and kv.n_free == 4
    kv.fork(0, 1)
    kv.truncate(0, 0)
    assert kv.compact() == []
    kv.extend(0, 1)
    kv.fork(0, 1, 1)
    assert kv.refs.tolist() == [2, 0, 0, 0]
    assert kv.extend(1, 1) == [(0, 1)] and kv.extend(0, 1) == []
    kv.truncate(0)
    assert kv.compact() == [(1, 0)] and kv.tables[1, 0] == 0 and kv.n_free == 3
