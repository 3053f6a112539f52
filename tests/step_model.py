"""Models in 64 bits of what stands around the attention and the experts: norms
and rotation of queries and keys, attention over any set of visible positions,
trees of drafts, routing, log probabilities; each with the bound on the library's
error.  Written from the definitions in include/moe_decode.h; they share no code
with the library."""
import numpy as np

from .kv_model import HALF, TOP

U = 2.0 ** -24      # half a step of fp32, relative


def rope(x, w, eps, positions, inv_freq, interleaved, factor, out):
    """x [rows][heads][D]: the output, and how far the library's may be off.

    The sum of squares (8 fused terms a lane, at most 5 levels across lanes) and
    its product with 1 / D and the addition of eps are off by 16 u relatively, its
    root by half that and one rounding, the reciprocal by one more: 10 u; the two
    products with weight and value: z is off by 12 u (without a norm by 0).  A
    cosine is off by 3 u (its argument, at most pi / 4, by one rounding, the
    series by its own roundings), times factor by 4 u factor; the pair's two
    products and their sum round once each."""
    rows, heads, D = x.shape
    z = x.astype(np.float64)
    cz = 0.0
    if w is not None:
        z = z / np.sqrt((z * z).mean(-1, keepdims=True) + eps) * w.astype(np.float64)
        cz = 12 * U
    y, tol = z.copy(), cz * np.abs(z)
    n = len(inv_freq)
    t = positions.astype(np.float64)[:, None] * inv_freq.astype(np.float64)
    c, s = factor * np.cos(t)[:, None], factor * np.sin(t)[:, None]
    a = np.arange(n) * 2 if interleaved else np.arange(n)
    b = a + 1 if interleaved else a + n
    y[..., a], y[..., b] = z[..., a] * c - z[..., b] * s, z[..., b] * c + z[..., a] * s
    tol[..., a] = tol[..., b] = (np.abs(z[..., a]) + np.abs(z[..., b])) * abs(factor) * (cz + 6 * U)
    return y, 1.05 * tol + HALF[out] * np.abs(y) + 1e-37


def tree_bits(parents):
    """Of one run: each token's ancestors and itself (numbers within the run),
    and how many ancestors it has; None where the chain is none."""
    out = []
    for i, p in enumerate(parents):
        if p == -1:
            out.append([i])
        elif 0 <= p < i and out[p] is not None:
            out.append(out[p] + [i])
        else:
            out.append(None)
    return out


def pack(bits, words):
    """Lists of bit numbers as signed 64-bit words."""
    m = np.zeros((len(bits), words), np.uint64)
    for r, row in enumerate(bits):
        for j in row or ():
            m[r, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return m.view(np.int64)


def visible(length, n, i, window, sinks, bits=None):
    """The positions that row i of a run of n sees; bits: its tree's tokens."""
    base = length - n
    if bits is None:
        p = base + i
        lo = max(0, p - window + 1) if window else 0
        see = set(range(lo, p + 1))
        if window:
            see |= set(range(min(sinks, p + 1)))
    else:
        bits = [j for j in bits if j < n]
        lo = max(0, base - max(window - len(bits), 0)) if window else 0
        see = set(range(lo, base)) | {base + j for j in bits}
        if window:
            see |= set(range(min(sinks, base)))
    return np.array(sorted(j for j in see if j >= 0), np.int64)


def attend(q, k, v, scale, seen, out, many):
    """One sequence, row i over the positions seen[i]: the output and the bound
    that kv_model.attention derives, with the tiles that hold those positions."""
    n, Hq, D = q.shape
    Hkv = k.shape[1]
    G, t = Hq // Hkv, TOP[out]
    o, tol = np.zeros(q.shape), np.zeros(q.shape)
    for i in range(n):
        at = seen[i]
        if not len(at):
            continue
        for h in range(Hq):
            kk, vv, qq = k[at, h // G], v[at, h // G], q[i, h].astype(np.float64)
            s = scale * (kk @ qq)
            e = np.exp(s - s.max())
            w = e / e.sum()
            o[i, h] = w @ vv
            A = abs(scale) * np.abs(qq).max() * np.abs(kk).sum(1).max()
            ds = A * (0.5 / t + 2 * U) + 12 * U * 2 * np.abs(s).max()
            V = w @ np.abs(vv)
            m = len(np.unique(at // 64)) * 64
            chain = (2 * m / 64 + 40) * U
            grid = np.abs(vv).sum(0) / t / e.sum() + len(at) / t / e.sum() * V
            if many:
                c = 2.0 ** -12 if out == "bf16" else 2.0 ** -23
                ds = A * (c + D * U) + 24 * U * np.abs(s).max()
                chain += c + m * U
                grid = m * 2.0 ** (-31 if out == "bf16" else -38) * np.abs(vv).max(0) / e.sum()
            tol[i, h] = 1.05 * (2 * (ds + 4 * U + chain) * V + grid) + HALF[out] * np.abs(o[i, h]) + 1e-37
    return o, tol


def route(logits, k, score, balance, groups, kept, best_two, renorm, scale):
    """One token: logits (fp32 values) -> experts, gates."""
    l = logits.astype(np.float64)
    E, n = len(l), len(l) // groups
    if score == "softmax":
        p = np.exp(l - l.max())
        p = p / p.sum()
    else:
        with np.errstate(over="ignore"):
            p = 1 / (1 + np.exp(-l))
    c = p if balance is None else p + balance.astype(np.float64)
    value = [sum(sorted(c[a:a + n], reverse=True)[:2 if best_two else 1]) for a in range(0, E, n)]
    held = sorted(range(groups), key=lambda g: (-value[g], g))[:kept]
    experts = [e for g in held for e in range(g * n, g * n + n)]
    won = sorted(experts, key=lambda e: (-c[e], e))[:k]
    g = p[won]
    if renorm:
        g = g / g.sum() if g.sum() else 0 * g
    return won, g * scale


def logprobs(x, scale):
    """Rows of fp32 values -> log probabilities, entropy, and the bounds on both.

    A term's z = (x - max) scale is off by 2 u |z|, its exp by that, one rounding of
    the exponent's product (u |z|) and the instruction's 2 u; a sum by k = 42 u and
    two roundings for each step of it (32 terms a thread and step, steps of 2048
    values at least, 6 levels, 4 waves).  With E = sum p |z|, E2 = sum p z^2: log Z
    by 3 u E + (k + 2) u, sum p z by 3 u E2 + (k + 4) u E and by E times what Z is off."""
    k = 42 + 2 * -(-(x.shape[1] + 7) // 2048)
    x = x.astype(np.float64)
    with np.errstate(invalid="ignore"):
        z = (x - x.max(1, keepdims=True)) * scale
        e = np.exp(z)
        Z = e.sum(1, keepdims=True)
        p, zz = e / Z, np.where(e > 0, z, 0.0)
        lp = z - np.log(Z)
        H = np.log(Z)[:, 0] - (p * zz).sum(1)
        E, E2 = (p * np.abs(zz)).sum(1), (p * zz * zz).sum(1)
    dz = 3 * U * E + (k + 2) * U
    return (lp, 1.1 * dz[:, None] + np.where(np.isfinite(lp), U * np.abs(lp), 0.0),
            H, 1.1 * (dz * (1 + E) + 3 * U * E2 + (k + 4) * U * E) + U * np.abs(H))


def top_ids(x, n):
    """The n largest of each row, equal ones by the lower id, a NaN the smallest."""
    x = np.asarray(x, np.float64) + 0.0
    out = []
    for row in x:
        order = sorted(range(len(row)), key=lambda i: (np.isnan(row[i]), -row[i] if row[i] == row[i] else 0.0, i))
        out.append(order[:n])
    return np.array(out, np.int32).reshape(len(x), n)
