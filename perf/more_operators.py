"""The operators of a step that checks drafted tokens, as they are measured: their
cases, inputs, plain forms, and the calls a program makes.

  rope     norms of queries and keys for each head, and their rotation by
           position, in one pass.
  attend   attention over the paged 8-bit cache where the new tokens are the
           nodes of a tree of drafts, or where a sliding window leaves the first
           tokens visible, or both.
  route    routing to experts: softmax or sigmoid scores, a bias that only the
           choice sees, groups, top-k, gates renormalised or not.
  logp     log probabilities of given tokens, the entropy and the top
           alternatives of rows of logits.

`run` computes the plain form, or makes the framework's calls where `own` is
true.  `exact` computes the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
F32, BF16 = "f32", "bf16"
DT = {F32: torch.float32, BF16: torch.bfloat16}
SIZE = {F32: 4, BF16: 2}


# ---- cases ---------------------------------------------------------------

def listed():
    return [
        # one decode token of the 1.1B-shaped dense block: latency only
        dict(name="rope_token", op="rope", T=1, Hq=32, Hkv=4, D=64, rot=64, pairs=False, norm=False, pos=4000, x=F32,
             y=F32),
        # a whole prompt's queries and keys, sliced out of the joint projection's output
        dict(name="rope_prompt", op="rope", T=8191, Hq=64, Hkv=8, D=128, rot=128, pairs=False, norm=True, pos=131071,
             x=BF16, y=BF16),
        # small trees of drafts of several sequences, wide heads
        dict(name="tree_verify", op="attend", S=9, q_max=12, kv_max=5000, Hq=16, Hkv=2, D=256, page=64, tree=True,
             window=0, sinks=0, x=BF16, y=F32),
        # larger trees on long contexts
        dict(name="tree_long", op="attend", S=2, q_max=61, kv_max=65535, Hq=32, Hkv=8, D=128, page=128, tree=True,
             window=0, sinks=0, x=F32, y=F32),
        # a decode batch that keeps to a window and the first tokens
        dict(name="sink_batch", op="attend", S=32, q_max=1, kv_max=30011, Hq=64, Hkv=8, D=128, page=64, tree=False,
             window=4096, sinks=4, x=BF16, y=BF16),
        # a prompt that does
        dict(name="sink_prompt", op="attend", S=1, q_max=4096, kv_max=9001, Hq=16, Hkv=4, D=128, page=64, tree=False,
             window=1024, sinks=100, x=BF16, y=BF16),
        # one token of the 128-expert layer
        dict(name="route_token", op="route", T=1, H=2048, E=128, k=8, score="softmax", balance=True, groups=1, kept=1,
             best_two=False, renorm=True, x=F32),
        # a 128-token chunk of the 256-expert layer
        dict(name="route_chunk", op="route", T=128, H=6144, E=256, k=8, score="sigmoid", balance=True, groups=8, kept=4,
             best_two=True, renorm=True, x=F32),
        # a whole prompt of it
        dict(name="route_prompt", op="route", T=8191, H=6144, E=256, k=8, score="sigmoid", balance=True, groups=8,
             kept=4, best_two=True, renorm=True, x=BF16),
        # one sampled token with its alternatives
        dict(name="logp_token", op="logp", rows=1, V=32000, given=1, top=5, scale=1.0, x=F32),
        # every node of some trees with its children, a vocabulary of odd size
        dict(name="logp_draft", op="logp", rows=288, V=131071, given=4, top=8, scale=1.25, x=BF16),
        # a prompt's own tokens
        dict(name="logp_prompt", op="logp", rows=4096, V=32000, given=1, top=0, scale=1.0, x=F32),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "attend", "route", "logp"])
    x = rng.choice([F32, BF16])
    if op == "rope":
        D = rng.choice([64, 80, 96, 128, 192, 256])
        Hkv = rng.choice([1, 2, 3, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 7, 8])
        T = max(1, min(_log(rng, 1, 16384), 8191 * 72 * 128 // (2 * (Hq + Hkv) * D)))
        return dict(op=op, T=T, Hq=Hq, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 16 * 8, 32]), pairs=rng.random() < 0.4,
                    norm=rng.random() < 0.7, pos=_log(rng, T, 1 << 20), x=x, y=rng.choice([F32, BF16]))
    if op == "route":
        E = rng.choice([8, 16, 60, 64, 128, 160, 256])
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0 and E // g >= 2])
        kept = rng.randint(1, groups)
        H = 256 * _log(rng, 1, 28)
        T = max(1, min(_log(rng, 1, 8191), 8191 * 6144 * 256 // (E * H)))
        return dict(op=op, T=T, H=H, E=E, k=rng.randint(1, min(8, kept * (E // groups))),
                    score=rng.choice(["softmax", "sigmoid"]), balance=rng.random() < 0.7, groups=groups, kept=kept,
                    best_two=rng.random() < 0.5, renorm=rng.random() < 0.7, x=x)
    if op == "logp":
        V = _log(rng, 100, 160000)
        rows = max(1, min(_log(rng, 1, 4096), 4096 * 16000 // V))
        return dict(op=op, rows=rows, V=V, given=rng.choice([0, 1, 1, 2, 5]), top=rng.choice([0, 1, 3, 5, 8, 20]),
                    scale=rng.choice([1.0, 0.7, 1.6]), x=x)
    D, page = rng.choice([64, 128, 256]), rng.choice([64, 128, 256])
    Hkv, G = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 7, 8, 16])
    tree = rng.random() < 0.6
    S, q_max = _log(rng, 1, 32), _log(rng, 1, 200 if tree else 1500)
    q_max = max(1, min(q_max, 4096 * 8 // (Hkv * G * S)))
    kv_max = max(q_max, min(_log(rng, 16, 65536), (1 << 27) // (S * Hkv * D * 2),
                            4096 * 1024 * 16 * 128 // (q_max * Hkv * G * S * D)))
    window = _log(rng, 1, 4096) if not tree or rng.random() < 0.3 else 0
    sinks = _log(rng, 1, 200) if window and (not tree or rng.random() < 0.5) else 0
    return dict(op=op, S=S, q_max=q_max, kv_max=kv_max, Hq=Hkv * G, Hkv=Hkv, D=D, page=page, tree=tree, window=window,
                sinks=sinks, x=x, y=rng.choice([F32, BF16]))


# ---- inputs --------------------------------------------------------------

def _lengths(c):
    """New and cached tokens of the sequences (host lists), the same for every
    seed: the first one has the largest of both, the others are spread below."""
    S = c["S"]
    u = torch.rand(2, S, generator=torch.Generator().manual_seed(137 * c["kv_max"] + c["q_max"])).tolist()
    nq = [max(1, int(round(c["q_max"] * (0.4 + 0.6 * a)))) for a in u[0]]
    kv = [max(n, int(round(c["kv_max"] * (0.1 + 0.9 * b)))) for n, b in zip(nq, u[1])]
    nq[0], kv[0] = c["q_max"], max(c["q_max"], c["kv_max"])
    return nq, kv


def _parents(c, h):
    """A tree of drafts for each sequence: token 0 is the last accepted one, the
    others hang on one of the six before them."""
    out = []
    for n in _lengths(c)[0]:
        u = torch.rand(n, generator=h).tolist()
        out.append([-1] + [max(0, i - 1 - int(6 * u[i])) for i in range(1, n)])
    return out


def _masks(parents):
    """Which tokens of its run each token sees, one bit each, 64 in a word."""
    words = max(-(-len(p) // 64) for p in parents)
    rows = []
    for p in parents:
        bits = []
        for i, q in enumerate(p):
            bits.append((bits[q] if q >= 0 else 0) | 1 << i)
        for b in bits:
            w = [b >> 64 * j & (1 << 64) - 1 for j in range(words)]
            rows.append([v - (1 << 64) if v >> 63 else v for v in w])
    return torch.tensor(rows, dtype=torch.int64)


def _cache(c, n_pages, g):
    """Codes and scales as a cache of keys and values near N(0, 1) holds them."""
    s = {}
    for name, shape in (("k", (n_pages, c["Hkv"], c["page"], c["D"])), ("v", (n_pages, c["Hkv"], c["D"], c["page"]))):
        codes = torch.empty(shape, dtype=torch.int8, device=DEV)
        flat = codes.view(-1)
        step = 1 << 27
        for a in range(0, flat.numel(), step):
            part = torch.randn(min(step, flat.numel() - a), generator=g, device=DEV)
            flat[a:a + step] = (part * 38).round_().clamp_(-127, 127).to(torch.int8)
        s[name] = codes
        s[name + "_scale"] = 0.02 + 0.015 * torch.rand(n_pages, c["Hkv"], generator=g, device=DEV)
    return s


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c = case
    g, h = torch.Generator(device=DEV).manual_seed(seed), torch.Generator().manual_seed(seed)

    def rn(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    s = {"case": c}
    if c["op"] == "rope":
        T, D, Hq, Hkv = c["T"], c["D"], c["Hq"], c["Hkv"]
        # the joint projection's output: queries, keys and values of a token in one row
        s["qkv"] = (rn(T, Hq + 2 * Hkv, D) * (1 + 0.5 * torch.rand(1, Hq + 2 * Hkv, 1, generator=g, device=DEV))
                    ).to(DT[c["x"]])
        s["q"], s["k"] = s["qkv"][:, :Hq], s["qkv"][:, Hq:Hq + Hkv]
        start = int(torch.randint(0, c["pos"] - T + 1, (1,), generator=h))
        s["positions"] = start + torch.arange(T, dtype=torch.int32, device=DEV)
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])).float().to(DEV)
        s["q_weight"] = 1 + 0.2 * rn(D) if c["norm"] else None
        s["k_weight"] = 1 + 0.2 * rn(D) if c["norm"] else None
        s["eps"] = 1e-6
        return s
    if c["op"] == "route":
        T, H, E = c["T"], c["H"], c["E"]
        s["x"] = rn(T, H).to(DT[c["x"]])
        s["Wr"] = rn(E, H) * (1.5 / math.sqrt(H))
        s["balance"] = (0.05 if c["score"] == "sigmoid" else 0.5 / E) * rn(E) if c["balance"] else None
        s["scale"] = 2.5 if c["score"] == "sigmoid" else 1.0
        return s
    if c["op"] == "logp":
        R, V = c["rows"], c["V"]
        # logits as a head leaves them: a broad bulk, and a few tokens far above it
        logits = 2 * rn(R, V)
        likely = torch.randint(0, V, (R, 8), generator=g, device=DEV)
        logits.scatter_add_(1, likely, 4 + 6 * torch.rand(R, 8, generator=g, device=DEV))
        s["logits"] = logits.to(DT[c["x"]])
        some = torch.randint(0, V, (R, max(1, c["given"])), generator=g, device=DEV)
        some[:, :1] = likely[:, :1]
        s["tokens"] = some[:, :c["given"]].int().contiguous() if c["given"] else None
        return s
    nq, kv = _lengths(c)
    need = [-(-n // c["page"]) for n in kv]
    order = torch.randperm(sum(need), generator=h, dtype=torch.int32)
    table = torch.zeros(c["S"], max(need), dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    starts = [0]
    for n in nq:
        starts.append(starts[-1] + n)
    s.update(q_start=_i32(starts), kv_len=_i32(kv), table=table.to(DEV), rows=starts[-1], q_max=c["q_max"],
             kv_max=max(kv), **_cache(c, sum(need), g))
    s["q"] = (1.3 * rn(starts[-1], c["Hq"], c["D"])).to(DT[c["x"]])
    s["masks"] = _masks(_parents(c, h)).to(DEV) if c["tree"] else None
    return s


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["T"] * (c["Hq"] + c["Hkv"]) * c["D"]
        return {"bytes": n * (SIZE[c["x"]] + SIZE[c["y"]]) + 4 * c["T"], "flops": 0}
    if c["op"] == "route":
        T, H, E = c["T"], c["H"], c["E"]
        return {"bytes": T * H * SIZE[c["x"]] + 4 * E * H + 8 * T * c["k"], "flops": 2 * T * H * E}
    if c["op"] == "logp":
        R = c["rows"]
        return {"bytes": R * (c["V"] * SIZE[c["x"]] + 8 * c["given"] + 4 + 8 * c["top"]), "flops": 0}
    nq, kv = _lengths(c)
    h = torch.Generator().manual_seed(0)
    parents = _parents(c, h) if c["tree"] else None
    read = pairs = 0        # cache positions read, and (query, key) pairs seen
    for i, (m, n) in enumerate(zip(nq, kv)):
        base = n - m
        w, k = c["window"] or n, min(c["sinks"], n)
        depth = []
        for j in range(m):      # how many tokens of the run each one sees
            depth.append(j + 1 if parents is None else 1 + (depth[parents[i][j]] if parents[i][j] >= 0 else 0))
        lo = [max(0, base - max(w - d, 0)) if parents is not None else max(0, base + j + 1 - w)
              for j, d in enumerate(depth)]
        first = min(lo)
        read += n - first + min(k, first)
        for j, a in enumerate(lo):
            run = depth[j] if parents is not None else 0
            end = base if parents is not None else base + j + 1
            pairs += run + end - a + min(k, a)
    return {"bytes": read * 2 * c["Hkv"] * c["D"] + sum(nq) * c["Hq"] * c["D"] * (SIZE[c["x"]] + SIZE[c["y"]]),
            "flops": 4 * pairs * c["Hq"] * c["D"]}


# ---- plain forms ---------------------------------------------------------

def _rope_one(s, x, weight):
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * weight
    # far positions: the angle needs 64 bits before its period is taken off
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    y = x.clone()
    if c["pairs"]:
        a, b = x[..., :rot:2], x[..., 1:rot:2]
        y[..., :rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :half], x[..., half:rot]
        y[..., :half], y[..., half:rot] = a * cos - b * sin, b * cos + a * sin
    return y.to(DT[c["y"]])


def _route(s):
    c = s["case"]
    # scores next to each other decide: 64 bits, the logits rounded once to 32
    l = (s["x"].double() @ s["Wr"].double().t()).float().double()
    if c["score"] == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-l))
    choice = p if s["balance"] is None else p + s["balance"].double()
    T, E, n = c["T"], c["E"], c["groups"]
    if c["kept"] < n:
        per = choice.view(T, n, E // n)
        best = torch.sort(per, dim=2, descending=True).values
        value = best[..., 0] + best[..., 1] if c["best_two"] else best[..., 0]
        keep = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :c["kept"]]
        held = torch.zeros(T, n, dtype=torch.bool, device=DEV).scatter_(1, keep, True)
        choice = choice.masked_fill(~held.repeat_interleave(E // n, 1), -math.inf)
    idx = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    gates = p.gather(1, idx)
    if c["renorm"]:
        gates = gates / gates.sum(1, keepdim=True)
    return {"idx": idx.int(), "gates": (gates * s["scale"]).float()}


def _logp(s):
    c = s["case"]
    x = s["logits"].float()
    z = x * c["scale"]
    z = z - z.amax(1, keepdim=True)
    e = torch.exp(z)
    total = e.sum(1, keepdim=True)
    norm = torch.log(total)
    out = {"entropy": (norm - (e * z).sum(1, keepdim=True) / total)[:, 0]}
    if s["tokens"] is not None:
        out["logprobs"] = z.gather(1, s["tokens"].long()) - norm
    if c["top"]:
        col = torch.arange(c["V"], device=DEV, dtype=torch.int32)
        left, ids = x.clone(), []
        for _ in range(c["top"]):      # the largest, the first where several are
            m = left.amax(1, keepdim=True)
            ids.append(torch.where(left == m, col, c["V"]).amin(1, keepdim=True))
            left.scatter_(1, ids[-1].long(), -math.inf)
        out["top_ids"] = torch.cat(ids, 1)
        out["top_logprobs"] = z.gather(1, out["top_ids"].long()) - norm
    return out


def _seen(s, S, nq, n):
    """Which cache positions each new token sees: [S][nq][n]."""
    c = s["case"]
    start, kv_len = s["q_start"].long(), s["kv_len"].long()
    count = start[1:] - start[:-1]
    i, j = torch.arange(nq, device=DEV), torch.arange(n, device=DEV)
    base = (kv_len - count)[:, None, None]
    if not c["tree"]:
        pos = base + i[:, None]
        seen = j <= pos
        if c["window"]:
            seen = seen & ((j > pos - c["window"]) | (j < c["sinks"]))
        return seen & (j < kv_len[:, None, None])
    take = (start[:-1, None] + i).clamp(max=s["rows"] - 1)
    bits = (s["masks"][take][..., None] >> torch.arange(64, device=DEV)) & 1
    bits = bits.flatten(2)[..., :nq].bool() & (i[None, None] < count[:, None, None])     # S nq nq
    seen = (j < base).expand(S, nq, n)
    if c["window"]:
        left = (c["window"] - bits.sum(2, keepdim=True)).clamp(min=0)
        seen = seen & ((j >= base - left) | (j < c["sinks"]))
    run = (j - base).clamp(0, nq - 1).expand(S, nq, n)
    return seen | (bits.gather(2, run) & (j >= base) & (j < kv_len[:, None, None]))


def _attend(s):
    c = s["case"]
    f = torch.float32
    S, Hkv, D, G, nq, n = c["S"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"], s["q_max"], s["kv_max"]
    pages = s["table"].long()
    k = (s["k"][pages].to(f) * s["k_scale"][pages][..., None, None]).transpose(1, 2)     # S Hkv pages page D
    v = (s["v"][pages].to(f) * s["v_scale"][pages][..., None, None]).permute(0, 2, 1, 4, 3)
    k, v = k.reshape(S, Hkv, -1, D)[:, :, :n], v.reshape(S, Hkv, -1, D)[:, :, :n]
    start = s["q_start"].long()
    take = (start[:-1, None] + torch.arange(nq, device=DEV)).clamp(max=s["rows"] - 1)
    q = s["q"][take].to(f).view(S, nq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(S, Hkv, G * nq, D)
    t = (q @ k.transpose(2, 3)).view(S, Hkv, G, nq, n).mul_(1 / math.sqrt(D))
    t.masked_fill_(~_seen(s, S, nq, n)[:, None, None], -math.inf)
    t -= t.amax(-1, keepdim=True).clamp(min=torch.finfo(f).min)
    t.exp_()
    total = t.sum(-1, keepdim=True)
    o = t.view(S, Hkv, G * nq, n) @ v
    o = o.view(S, Hkv, G, nq, D) / torch.where(total > 0, total, torch.ones_like(total))
    r = torch.arange(s["rows"], device=DEV)
    seq = torch.searchsorted(s["q_start"][1:].contiguous(), r.int(), right=True)
    return o.permute(0, 3, 1, 2, 4)[seq, r - start[seq]].reshape(s["rows"], c["Hq"], D).to(DT[c["y"]])


# ---- the framework's calls -----------------------------------------------

def _handles(s):
    """What a program keeps between calls: the descriptors of its cache, its
    batch and its routing."""
    import moe_decode_amd as md
    c = s["case"]
    if c["op"] == "attend":
        s["own"] = md.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["batch"] = md.KVBatch(s["q_start"], s["kv_len"], s["table"], s["q_max"], s["kv_max"])
    else:
        s["own"] = md.Routing(c["k"], score=c["score"], balance=s["balance"], groups=c["groups"], groups_kept=c["kept"],
                              best_two=c["best_two"], renorm=c["renorm"], scale=s["scale"])


def _own(s):
    import moe_decode_amd as md
    c = s["case"]
    if c["op"] == "rope":
        return md.qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], q_weight=s["q_weight"],
                               k_weight=s["k_weight"], eps=s["eps"], interleaved=c["pairs"], out_dtype=DT[c["y"]])
    if c["op"] == "logp":
        r = md.token_logprobs(s["logits"], tokens=s["tokens"], top=c["top"], scale=c["scale"])
        return {name: t for name, t in r._asdict().items() if t is not None}
    if "own" not in s:
        _handles(s)
    if c["op"] == "route":
        idx, gates = md.moe_route(s["x"], s["Wr"], s["own"])
        return {"idx": idx, "gates": gates}
    return md.kv_attention(s["own"], s["batch"], s["q"], window=c["window"], sinks=c["sinks"], tree=s["masks"],
                           out_dtype=DT[c["y"]])


def run(state):
    s = state
    if own:
        return _own(s)
    op = s["case"]["op"]
    if op == "rope":
        return _rope_one(s, s["q"], s["q_weight"]), _rope_one(s, s["k"], s["k_weight"])
    return {"route": _route, "logp": _logp, "attend": _attend}[op](s)


# ---- the definitions in 64 bits ------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "route": _exact_route, "logp": _exact_logp, "attend": _exact_attend}[case["op"]](s)


def _exact_rope(s):
    """Pairs of channels as complex numbers, turned by exp(i angle)."""
    c = s["case"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       torch.outer(s["positions"].double(), s["inv_freq"].double()))[:, None]
    out = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        x = x.double()
        if w is not None:
            size = torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / c["D"]
            x = x / torch.sqrt(size + s["eps"]) * w.double()
        head, tail = x[..., :c["rot"]], x[..., c["rot"]:]
        pair = head.unflatten(-1, (-1, 2)) if c["pairs"] else head.unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        z = z.flatten(-2) if c["pairs"] else z.transpose(-1, -2).flatten(-2)
        out.append(torch.cat([z, tail], -1))
    return tuple(out)


def _exact_route(s):
    """Token by token on the host, from the logits in 64 bits."""
    c = s["case"]
    logits = torch.stack([torch.mv(s["Wr"].double(), row) for row in s["x"].double()]).float().cpu().numpy()
    bias = np.zeros(c["E"]) if s["balance"] is None else s["balance"].double().cpu().numpy()
    n = c["E"] // c["groups"]
    ids, gates = [], []
    for l in logits.astype(np.float64):
        if c["score"] == "softmax":
            p = np.exp(l - l.max())
            p = p / p.sum()
        else:
            p = 1.0 / (1.0 + np.exp(-l))
        choice = p + bias
        value = [sum(sorted(choice[a:a + n])[::-1][:2 if c["best_two"] else 1]) for a in range(0, c["E"], n)]
        held = sorted(range(c["groups"]), key=lambda a: (-value[a], a))[:c["kept"]]
        experts = [e for a in held for e in range(a * n, a * n + n)]
        won = sorted(experts, key=lambda e: (-choice[e], e))[:c["k"]]
        ids.append(won)
        gates.append(p[won] / (p[won].sum() if c["renorm"] else 1.0) * s["scale"])
    return {"idx": torch.tensor(ids, dtype=torch.int32), "gates": torch.tensor(np.stack(gates))}


def _exact_logp(s):
    """A block of rows at a time; alternatives by a stable sort."""
    c = s["case"]
    parts = []
    for a in range(0, c["rows"], 256):
        x = s["logits"][a:a + 256].double()
        lp = torch.log_softmax(x * c["scale"], 1)
        part = {"entropy": torch.special.entr(lp.exp()).sum(1)}
        if s["tokens"] is not None:
            part["logprobs"] = torch.take_along_dim(lp, s["tokens"][a:a + 256].long(), 1)
        if c["top"]:
            part["top_ids"] = torch.argsort(x, dim=1, descending=True, stable=True)[:, :c["top"]].int()
            part["top_logprobs"] = torch.take_along_dim(lp, part["top_ids"].long(), 1)
        parts.append(part)
    return {name: torch.cat([p[name] for p in parts]) for name in parts[0]}


def _exact_attend(s):
    """One sequence and key head after another, a block of new tokens at a time."""
    c = s["case"]
    G, D, page = c["Hq"] // c["Hkv"], c["D"], c["page"]
    starts, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    masks = s["masks"].tolist() if c["tree"] else None
    out = torch.zeros(s["rows"], c["Hq"], D, dtype=torch.float64, device=DEV)
    for i, n in enumerate(lens):
        m = starts[i + 1] - starts[i]
        hide = torch.zeros(m, n, dtype=torch.bool)
        key = torch.arange(n)
        for j in range(m):
            if c["tree"]:
                mine = [n - m + b for b in range(m) if masks[starts[i] + j][b // 64] >> b % 64 & 1]
                hide[j, n - m:] = True
                if c["window"]:
                    hide[j, :max(0, n - m - max(0, c["window"] - len(mine)))] = True
                hide[j, :min(c["sinks"], n - m)] = False
                hide[j, mine] = False
            else:
                at = n - m + j
                hide[j] = key > at
                if c["window"]:
                    hide[j] |= (key <= at - c["window"]) & (key >= c["sinks"])
        hide = hide.to(DEV)
        ids = s["table"][i, : -(-n // page)].long()
        for h in range(c["Hkv"]):
            k = (s["k"][ids, h].double() * s["k_scale"][ids, h].double()[:, None, None]).reshape(-1, D)[:n]
            v = s["v"][ids, h].double() * s["v_scale"][ids, h].double()[:, None, None]
            v = v.transpose(1, 2).reshape(-1, D)[:n]
            some = max(1, (1 << 26) // (G * n))
            for a in range(0, m, some):
                b = min(a + some, m)
                rows = slice(starts[i] + a, starts[i] + b)
                q = s["q"][rows, h * G:(h + 1) * G].double().reshape(-1, D)
                score = torch.mm(q, k.t().contiguous()) / math.sqrt(D)
                score[hide[a:b].repeat_interleave(G, 0)] = -math.inf
                out[rows, h * G:(h + 1) * G] = torch.mm(torch.softmax(score, 1), v).view(b - a, G, D)
    return out
