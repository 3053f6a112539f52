"""Models of the 8-bit attention block in numpy: the codes of activations, the
append into a paged cache, attention in 64 bits with the bound on the library's
error, and the page bookkeeping.  Written from the definitions in
include/moe_decode.h; they share no code with the library."""
import numpy as np

TOP = {"f32": 8355711.0, "bf16": 32639.0}     # integers of a query row and of a softmax weight, by output type
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # half a step of a rounded output, relative


def step_of(a):
    """max / 127 rounded to fp32 (the fp64 quotient never lies so near a tie of
    fp32 that rounding twice could differ)."""
    return np.float32(np.float64(a) / 127.0)


def codes_of(x, s):
    """x / s to the nearest integer, ties to even, -127..127; 0 where s is 0.
    The fp64 quotient of two fp32 values equals k + 1/2 only if the exact one
    does: (k + 1/2) s has at most 32 bits."""
    x, s = np.broadcast_arrays(np.asarray(x, np.float64), np.asarray(s, np.float64))
    out = np.zeros(x.shape)
    ok = s > 0
    out[ok] = np.clip(np.rint(x[ok] / s[ok]), -127, 127)
    return out.astype(np.int8)


class Cache:
    """One layer's cache; keys and values both held as [page][head][token][channel]."""

    def __init__(self, n_pages, heads, page, dim, rng):
        shape = (n_pages, heads, page, dim)
        self.page = page
        self.c = {n: rng.integers(-127, 128, size=shape).astype(np.int8) for n in "kv"}
        self.s = {n: rng.uniform(0.01, 0.03, size=shape[:2]).astype(np.float32) for n in "kv"}

    def append(self, table, first, rows):
        """rows: {"k": [n][head][channel] fp32, "v": ...} at positions first..."""
        n, P = len(rows["k"]), self.page
        at = max(0, -first)
        while at < n:
            pos = first + at
            take = min(n - at, P - pos % P)
            pg, lo = table[pos // P], pos % P
            for name in "kv":
                x = rows[name][at:at + take]
                for h in range(x.shape[1]):
                    self._one(name, pg, h, lo, x[:, h])
            at += take

    def _one(self, name, pg, h, lo, x):
        c, was = self.c[name][pg, h], (self.s[name][pg, h] if lo else np.float32(0))
        if not np.isfinite(x).all() or not np.isfinite(was):
            self.s[name][pg, h] = np.nan
            c[lo:lo + len(x)] = 0
            return
        need, now, up = step_of(np.abs(x).max()), was, 0
        if was == 0:
            now = need
        else:
            while now < need:
                now, up = np.float32(now * np.float32(2)), up + 1
        if up:
            c[:lo] = np.rint(c[:lo].astype(np.float64) / 2.0 ** up)
        c[lo:lo + len(x)] = codes_of(x, now)
        self.s[name][pg, h] = now

    def values(self, name, table, n):
        """[token][head][channel] in 64 bits."""
        ids = np.asarray(table[: -(-n // self.page)], dtype=np.int64)
        v = self.c[name][ids].astype(np.float64) * self.s[name][ids].astype(np.float64)[..., None, None]
        return v.transpose(0, 2, 1, 3).reshape(-1, v.shape[1], v.shape[3])[:n]


def attention(q, k, v, scale, causal, window, out, many=False):
    """One sequence: q [n][Hq][D], k, v [len][Hkv][D] in 64 bits.  Returns the
    output and how far the library's may be off.

    With u = 2^-24 (fp32) and the integers' top value t (TOP):
    - a query's channel is off by half an integer step, plus two fp32 roundings
      of the factor and product, together at most 2 |n| u <= 2 t u steps, so by
      (1/2 + 2 t u) M / t, M the row's largest magnitude; a score by that times
      scale sum |k|, and relatively by its own fp32 roundings (the joins' three,
      the factors' five, the product and the subtraction of the maximum: 10 u,
      and the last one is relative to score - max, at most twice the largest
      score);
    - exp2 is good to 2 u relatively, so a weight is off by the factor
      1 + e, e = score error + 4 u, and its grid by 1/2 + (its fma) < 1 step of 1 / t;
    - both sums are chains of one product and one addition a tile, and 16 terms
      in a lane, 2 levels across lanes, 4 waves and the splits: (2 tiles + 40) u.
    The quotient takes both sums' errors.

    many (over 64 columns, max_q * Hq / Hkv): both products in f16 with fp32
    sums.  A query's channel and a weight are off relatively by c = 2^-12 (bf16
    outputs), or 2^-23 where a second f16 holds the first one's remainder (13 of
    24 bits, rounded to 11), with floors (2^-25 of 2^14) that the weights show
    as n 2^-38 max |v| (bf16 outputs: of 2^7, n 2^-31 max |v|); a sum of D products is off by D u of its terms' sizes, one
    of n weights by n u."""
    n, Hq, D = q.shape
    L, Hkv = k.shape[0], k.shape[1]
    G, u, t = Hq // Hkv, 2.0 ** -24, TOP[out]
    o, tol = np.zeros(q.shape), np.zeros(q.shape)
    for i in range(n):
        p = L - n + i
        hi = p + 1 if causal else L
        lo = max(0, p - window + 1) if window else 0
        if hi <= lo:
            continue
        for h in range(Hq):
            kk, vv, qq = k[lo:hi, h // G], v[lo:hi, h // G], q[i, h].astype(np.float64)
            s = scale * (kk @ qq)
            e = np.exp(s - s.max())
            w = e / e.sum()
            o[i, h] = w @ vv
            A = abs(scale) * np.abs(qq).max() * np.abs(kk).sum(1).max()
            ds = A * (0.5 / t + 2 * u) + 12 * u * 2 * np.abs(s).max()
            V = w @ np.abs(vv)
            chain = (2 * (hi - lo) / 64 + 40) * u
            grid = np.abs(vv).sum(0) / t / e.sum() + (hi - lo) / t / e.sum() * V
            if many:
                c = 2.0 ** -12 if out == "bf16" else 2.0 ** -23
                ds = A * (c + D * u) + 24 * u * np.abs(s).max()
                chain += c + (hi - lo) * u
                grid = (hi - lo) * 2.0 ** (-31 if out == "bf16" else -38) * np.abs(vv).max(0) / e.sum()
            tol[i, h] = 1.05 * (2 * (ds + 4 * u + chain) * V + grid) + HALF[out] * np.abs(o[i, h]) + 1e-37
    return o, tol


def many_columns(max_q, G, D, out):
    """Which of the two forms a call takes."""
    return max_q * G > (768 if D == 256 and out == "f32" else 64)


class Pages:
    """The page bookkeeping by plain sets: which table names which page."""

    def __init__(self, n, page):
        self.n, self.page, self.tables = n, page, {}

    def used(self):
        return {p for t in self.tables.values() for p in t}

    def refs(self, p):
        return sum(p in t for t in self.tables.values())

    def take(self):
        free = sorted(set(range(self.n)) - self.used())
        return free[0] if free else None
