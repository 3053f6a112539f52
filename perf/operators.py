"""The 8-bit attention block's operators as they are measured: their cases,
inputs, plain forms, and the calls a program makes.

  linear   y = Q(x) W^T (+ bias): activations rounded to 8-bit integers with a
           scale for each token, int8 weights with a scale for each output
           channel, the product summed in integers.
  attend   attention of new queries over a paged cache whose keys and values
           are 8-bit integers with one scale for each page and head.
  append   new keys and values written into that cache: a page's scale is set
           by what first reaches it and grows by powers of two.
  copy     pages of the cache copied to other pages (a fork's first write to a
           shared page, a compaction).

`run` computes the plain form, or makes the framework's calls where `own` is
true.  `exact` computes the definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
F32, BF16 = "f32", "bf16"
DT = {F32: torch.float32, BF16: torch.bfloat16}


# ---- cases ---------------------------------------------------------------

def listed():
    return [
        # the key projection of a 1.1B-shaped dense block, one decode token
        dict(name="linear_token", op="linear", T=1, N=256, K=2048, x=F32, y=F32, bias=False),
        # a 128-token chunk through the output projection of a hidden-6144 layer
        dict(name="linear_chunk", op="linear", T=128, N=6144, K=6144, x=F32, y=F32, bias=True),
        # a whole prompt through the up projection of the 1.1B-shaped block's width class, odd token count
        dict(name="linear_prompt", op="linear", T=8191, N=5632, K=6144, x=BF16, y=BF16, bias=False),
        # one token on a short context: the 1.1B-shaped block's heads, latency only
        dict(name="attend_token", op="attend", S=1, q_max=1, kv_max=97, Hq=32, Hkv=4, D=64, page=64, causal=True,
             window=0, x=F32, y=F32),
        # a decode batch of ragged contexts
        dict(name="attend_batch", op="attend", S=32, q_max=1, kv_max=8190, Hq=64, Hkv=8, D=128, page=64,
             causal=True, window=0, x=BF16, y=BF16),
        # two decode tokens on very long contexts
        dict(name="attend_long", op="attend", S=2, q_max=1, kv_max=131071, Hq=32, Hkv=8, D=128, page=128,
             causal=True, window=0, x=F32, y=F32),
        # draft tokens checked by several sequences, wide heads, a sliding window
        dict(name="attend_verify", op="attend", S=9, q_max=7, kv_max=5000, Hq=16, Hkv=2, D=256, page=64,
             causal=True, window=1024, x=BF16, y=F32),
        # a prompt, causal, with a part of it already in the cache
        dict(name="attend_prompt", op="attend", S=1, q_max=4096, kv_max=5003, Hq=16, Hkv=4, D=128, page=64,
             causal=True, window=0, x=BF16, y=BF16),
        # one new token for each sequence of a decode batch
        dict(name="append_batch", op="append", S=64, q_max=1, kv_max=2049, Hkv=8, D=128, page=64, x=F32),
        # a prompt's keys and values
        dict(name="append_prompt", op="append", S=3, q_max=8192, kv_max=8200, Hkv=8, D=128, page=128, x=BF16),
        # the last, shared pages of a few forked sequences
        dict(name="copy_fork", op="copy", pages=64, pairs=7, Hkv=4, D=64, page=64),
        # a compaction of a large cache
        dict(name="copy_compact", op="copy", pages=6000, pairs=2001, Hkv=8, D=128, page=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "attend", "append", "copy"])
    x = rng.choice([F32, BF16])
    if op == "linear":
        T, K = _log(rng, 1, 8191), 256 * _log(rng, 1, 64)
        N = _log(rng, 1, max(1, min(20000, 8191 * 5632 * 6144 // (T * K))))
        return dict(op=op, T=T, N=N, K=K, x=x, y=rng.choice([F32, BF16]), bias=rng.random() < 0.5)
    D, page = rng.choice([64, 128, 256]), rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    if op == "copy":
        pairs = _log(rng, 1, 1500)
        return dict(op=op, pages=2 * pairs + rng.randint(0, 500), pairs=pairs, Hkv=Hkv, D=D, page=page)
    S, q_max = _log(rng, 1, 48), _log(rng, 1, 2048)
    if op == "append":
        q_max = max(1, min(q_max, 16384 // S))
        return dict(op=op, S=S, q_max=q_max, kv_max=q_max + rng.randint(0, 1000), Hkv=Hkv, D=D, page=page, x=x)
    G = rng.choice([1, 2, 3, 4, 7, 8, 16])
    # what a pass computes stays within the prompt's, what it reads within the long contexts'
    q_max = max(1, min(q_max, 4096 * 16 // (Hkv * G * S)))
    kv_max = max(q_max, min(_log(rng, 16, 65536), (1 << 28) // (S * Hkv * D * 2),
                            4096 * 4096 * 16 * 128 // (q_max * Hkv * G * S * D)))
    causal = rng.random() < 0.75
    window = _log(rng, 1, 4096) if causal and rng.random() < 0.3 else 0
    return dict(op=op, S=S, q_max=q_max, kv_max=kv_max, Hq=Hkv * G, Hkv=Hkv, D=D, page=page, causal=causal,
                window=window, x=x, y=rng.choice([F32, BF16]))


# ---- inputs --------------------------------------------------------------

def _lengths(c):
    """Query and cache lengths of the sequences (host lists), the same for every
    seed: the first one has the largest of both, the others are spread below."""
    S = c["S"]
    u = torch.rand(2, S, generator=torch.Generator().manual_seed(131 * c["kv_max"] + c["q_max"])).tolist()
    nq = [max(1, int(round(c["q_max"] * (0.4 + 0.6 * a)))) for a in u[0]]
    kv = [max(n, int(round(c["kv_max"] * (0.1 + 0.9 * b)))) for n, b in zip(nq, u[1])]
    nq[0], kv[0] = c["q_max"], max(c["q_max"], c["kv_max"])
    return nq, kv


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
    if c["op"] == "linear":
        T, N, K = c["T"], c["N"], c["K"]
        x = rn(T, K) * torch.exp(0.5 * rn(T, 1))
        x[:, :: max(1, K // 6)] *= 8.0      # a few channels far above the others, as hidden states have
        s["x"] = x.to(DT[c["x"]])
        s["w"] = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
        s["w_scale"] = 1e-3 + 9e-3 * torch.rand(N, generator=g, device=DEV)
        s["bias"] = rn(N) if c["bias"] else None
        return s
    if c["op"] == "copy":
        order = torch.randperm(c["pages"], generator=h)[: 2 * c["pairs"]].tolist()
        s["src"], s["dst"] = order[: c["pairs"]], order[c["pairs"]:]
        s["pairs"] = _i32(order).view(2, -1).long()
        return {**s, **_cache(c, c["pages"], g)}
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
    if c["op"] == "attend":
        s["q"] = (1.3 * rn(starts[-1], c["Hq"], c["D"])).to(DT[c["x"]])
    else:
        s["new_k"] = rn(starts[-1], c["Hkv"], c["D"]).to(DT[c["x"]])
        s["new_v"] = rn(starts[-1], c["Hkv"], c["D"]).to(DT[c["x"]])
        P = (c["q_max"] - 1) // c["page"] + 2     # pages that q_max tokens can touch
        start = [b - a for a, b in zip(nq, kv)]
        s["touched"] = _i32([int(table[i, p]) for i in range(c["S"])
                             for p in range(start[i] // c["page"], (kv[i] - 1) // c["page"] + 1)])
        s["pages_touched"] = P
    return s


def work(case):
    c = case
    e = {F32: 4, BF16: 2}
    if c["op"] == "linear":
        T, N, K = c["T"], c["N"], c["K"]
        return {"bytes": T * K * e[c["x"]] + N * K + 4 * N * (2 if c["bias"] else 1) + T * N * e[c["y"]],
                "flops": 2 * T * N * K}
    if c["op"] == "copy":
        return {"bytes": c["pairs"] * 2 * c["Hkv"] * (2 * c["page"] * c["D"] + 8), "flops": 0}
    nq, kv = _lengths(c)
    if c["op"] == "append":
        # the new rows read, their codes written, and the touched pages read back as fp32 values
        pages = sum((n - 1) // c["page"] - (n - m) // c["page"] + 1 for m, n in zip(nq, kv))
        return {"bytes": 2 * c["Hkv"] * c["D"] * (sum(nq) * (e[c["x"]] + 1) + pages * c["page"] * (1 + 4)), "flops": 0}
    read = pairs = 0        # cache positions read, and (query, key) pairs seen
    for m, n in zip(nq, kv):
        if not c["causal"]:
            read, pairs = read + n, pairs + m * n
            continue
        w = c["window"] or n
        read += min(n, m + w - 1)
        pairs += sum(min(p, w) for p in range(n - m + 1, n + 1))
    return {"bytes": read * 2 * c["Hkv"] * c["D"] + sum(nq) * c["Hq"] * c["D"] * (e[c["x"]] + e[c["y"]]),
            "flops": 4 * pairs * c["Hq"] * c["D"]}


# ---- plain forms ---------------------------------------------------------

def _codes(x, s):
    """x in steps of s as integers in -127..127, ties to even; in 64 bits, since
    a quotient may lie next to a border."""
    q = (x.double() / torch.where(s > 0, s, torch.ones_like(s)).double()).round().clamp(-127, 127)
    return torch.where(s > 0, q, torch.zeros_like(q))


def _step(x, dims):
    """The step that takes the largest magnitude to 127."""
    return (x.double().abs().amax(dims, keepdim=True) / 127).float()


def _linear(s):
    xs = _step(s["x"], 1)
    y = _codes(s["x"], xs).float() @ s["w"].float().t()
    y = y * xs * s["w_scale"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(DT[s["case"]["y"]])


def _rows_of(s):
    """The sequence of each query row, and its place among that sequence's."""
    r = torch.arange(s["rows"], device=DEV)
    seq = torch.searchsorted(s["q_start"][1:].contiguous(), r.int(), right=True)
    return seq, r - s["q_start"].long()[seq]


def _attend(s, f=torch.float32):
    c = s["case"]
    S, Hkv, D, G, nq, n = c["S"], c["Hkv"], c["D"], c["Hq"] // c["Hkv"], s["q_max"], s["kv_max"]
    pages = s["table"].long()
    k = (s["k"][pages].to(f) * s["k_scale"][pages][..., None, None].to(f)).transpose(1, 2)     # S Hkv pages page D
    v = (s["v"][pages].to(f) * s["v_scale"][pages][..., None, None].to(f)).permute(0, 2, 1, 4, 3)
    k, v = k.reshape(S, Hkv, -1, D)[:, :, :n], v.reshape(S, Hkv, -1, D)[:, :, :n]
    start, kv_len = s["q_start"].long(), s["kv_len"].long()
    count = start[1:] - start[:-1]
    i = torch.arange(nq, device=DEV)
    take = (start[:-1, None] + i).clamp(max=s["rows"] - 1)
    q = s["q"][take].to(f).view(S, nq, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(S, Hkv, G * nq, D)
    t = (q @ k.transpose(2, 3)).view(S, Hkv, G, nq, n).mul_(1 / math.sqrt(D))
    j = torch.arange(n, device=DEV)
    seen = (j < kv_len[:, None])[:, None, :]
    if c["causal"]:
        pos = (kv_len - count)[:, None] + i
        seen = seen & (j <= pos[..., None])
        if c["window"]:
            seen = seen & (j > pos[..., None] - c["window"])
    t.masked_fill_(~seen.expand(S, nq, n)[:, None, None], -math.inf)
    t -= t.amax(-1, keepdim=True).clamp(min=torch.finfo(f).min)
    t.exp_()
    total = t.sum(-1, keepdim=True)
    o = t.view(S, Hkv, G * nq, n) @ v
    o = o.view(S, Hkv, G, nq, D) / torch.where(total > 0, total, torch.ones_like(total))
    seq, at = _rows_of(s)
    return o.permute(0, 3, 1, 2, 4)[seq, at].reshape(s["rows"], c["Hq"], D)


def _append_one(s, name):
    """Writes the new rows into the pages that they touch; the values that those
    pages hold then, as [pages][Hkv][page][D]."""
    c = s["case"]
    page, new, codes, scale = c["page"], s["new_" + name], s[name], s[name + "_scale"]
    start, kv_len = s["q_start"].long(), s["kv_len"].long()
    first = kv_len - (start[1:] - start[:-1])
    # the pages of a sequence; past its last one, that one again (and so the same values)
    j = torch.minimum(first[:, None] // page + torch.arange(s["pages_touched"], device=DEV), (kv_len[:, None] - 1) // page)
    ids = s["table"].long().gather(1, j)
    pos = (j * page)[..., None] + torch.arange(page, device=DEV)
    is_old, is_new = pos < first[:, None, None], pos < kv_len[:, None, None]
    is_new = is_new & ~is_old
    take = (start[:-1, None, None] + pos - first[:, None, None]).clamp(0, s["rows"] - 1)
    x = new[take].float().transpose(2, 3) * is_new[:, :, None, :, None]         # S P Hkv page D
    old = codes[ids] if name == "k" else codes[ids].transpose(3, 4)
    was = scale[ids][..., None, None] * is_old.any(-1)[:, :, None, None, None]
    need = _step(x, (3, 4))
    a, b = torch.frexp(was), torch.frexp(need)
    up = torch.where((was > 0) & (need > was), b[1] - a[1] + (b[0] > a[0]).int(), torch.zeros_like(a[1]))
    now = torch.where(was > 0, torch.ldexp(was, up), need)
    kept = torch.ldexp(old.float(), -up).round()
    # a slot that no token has reached keeps its code
    q = torch.where(is_new[:, :, None, :, None], _codes(x, now).float(),
                    torch.where(is_old[:, :, None, :, None], kept, old.float())).to(torch.int8)
    codes[ids] = q if name == "k" else q.transpose(3, 4)
    scale[ids] = now[..., 0, 0]
    t = s["touched"].long()
    got = codes[t] if name == "k" else codes[t].transpose(2, 3)
    return got.float() * scale[t][..., None, None]


def _append(s):
    return {name: _append_one(s, name) for name in ("k", "v")}


def _copy(s):
    src, dst = s["pairs"]
    for name in ("k", "v", "k_scale", "v_scale"):
        s[name][dst] = s[name][src]
    return {name: s[name] for name in ("k", "v", "k_scale", "v_scale")}


# ---- the framework's calls -----------------------------------------------

def _handles(s):
    """What a program keeps between calls: the descriptors of its weights, its
    cache and its batch."""
    import moe_decode_amd as md
    c = s["case"]
    if c["op"] == "linear":
        s["own"] = md.DevQMatrix("i8_row", c["N"], c["K"], s["w"].view(-1), s["w_scale"])
        return md
    s["own"] = md.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if c["op"] in ("attend", "append"):
        s["batch"] = md.KVBatch(s["q_start"], s["kv_len"], s["table"], s["q_max"], s["kv_max"])
    return md


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import moe_decode_amd as md
        if "own" not in s:
            _handles(s)
        if op == "linear":
            return md.i8_linear(s["own"], s["x"], bias=s["bias"], out_dtype=DT[s["case"]["y"]])
        if op == "attend":
            return md.kv_attention(s["own"], s["batch"], s["q"], causal=s["case"]["causal"],
                                   window=s["case"]["window"], out_dtype=DT[s["case"]["y"]])
        if op == "append":
            md.kv_append(s["own"], s["batch"], s["new_k"], s["new_v"])
            k, v = md.kv_read_pages(s["own"], s["touched"])
            return {"k": k, "v": v}
        md.kv_copy_pages(s["own"], s["src"], s["dst"])
        return {name: s[name] for name in ("k", "v", "k_scale", "v_scale")}
    if op == "linear":
        return _linear(s)
    if op == "attend":
        return _attend(s).to(DT[s["case"]["y"]])
    return _append(s) if op == "append" else _copy(s)


# ---- the definitions in 64 bits ------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        x = s["x"].double()
        step = (x.abs().max(1).values / 127).float().double()[:, None]
        whole = torch.round(x / torch.where(step == 0, torch.ones_like(step), step)).clamp(-127, 127)
        y = torch.mm(whole, s["w"].double().t().contiguous())
        y = y * step * s["w_scale"].double()[None]
        return y if s["bias"] is None else y + s["bias"].double()
    if case["op"] == "copy":
        moved = {"k": None, "v": None}
        for name in ("k_scale", "v_scale"):
            t = s[name].tolist()
            for a, b in zip(s["src"], s["dst"]):
                t[b] = t[a]
            moved[name] = torch.tensor(t, dtype=torch.float64)
        return moved
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)


def _exact_append(s):
    """One page after another: its earlier codes halved as often as its scale
    doubles, then the new tokens."""
    page = s["case"]["page"]
    starts, lens, table = s["q_start"].tolist(), s["kv_len"].tolist(), s["table"].tolist()
    out = {"k": [], "v": []}
    for i, n in enumerate(lens):
        first = n - (starts[i + 1] - starts[i])
        for p in range(first // page, (n - 1) // page + 1):
            lo, hi = max(first, p * page), min(n, (p + 1) * page)
            rows, at = slice(starts[i] + lo - first, starts[i] + hi - first), slice(lo - p * page, hi - p * page)
            for name in ("k", "v"):
                held = s[name][table[i][p]].double()
                held = held.clone() if name == "k" else held.transpose(1, 2).clone()
                x = s["new_" + name][rows].double().transpose(0, 1)
                need = (x.abs().amax((1, 2)) / 127).float().double()
                if at.start:
                    step = s[name + "_scale"][table[i][p]].double()
                    while bool((need > step).any()):
                        twice = need > step
                        step = torch.where(twice, 2 * step, step)
                        held = torch.where(twice[:, None, None], held / 2, held)
                    held[:, : at.start] = held[:, : at.start].round()
                    # what no token has reached is outside: its codes stay as they were
                    raw = s[name][table[i][p]].double()
                    held[:, at.stop:] = (raw if name == "k" else raw.transpose(1, 2))[:, at.stop:]
                else:
                    step = need
                held[:, at] = (x / torch.where(step == 0, torch.ones_like(step), step)[:, None, None]).round().clamp(-127, 127)
                out[name].append(held * step[:, None, None])
    return {name: torch.stack(v) for name, v in out.items()}


def _exact_attend(s):
    """One sequence and key head after another, a block of rows at a time."""
    c = s["case"]
    G, D, page = c["Hq"] // c["Hkv"], c["D"], c["page"]
    starts, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    if sum((b - a) * n for a, b, n in zip(starts, starts[1:], lens)) * c["Hq"] * D > 3e12:
        return None
    out = torch.zeros(s["rows"], c["Hq"], D, dtype=torch.float64, device=DEV)
    for i, n in enumerate(lens):
        ids = s["table"][i, : -(-n // page)].long()
        for h in range(c["Hkv"]):
            k = (s["k"][ids, h].double() * s["k_scale"][ids, h].double()[:, None, None]).reshape(-1, D)[:n]
            v = s["v"][ids, h].double() * s["v_scale"][ids, h].double()[:, None, None]
            v = v.transpose(1, 2).reshape(-1, D)[:n]
            some = max(1, (1 << 26) // (G * n))
            for a in range(starts[i], starts[i + 1], some):
                b = min(a + some, starts[i + 1])
                q = s["q"][a:b, h * G:(h + 1) * G].double().reshape(-1, D)
                score = torch.mm(q, k.t().contiguous()) / math.sqrt(D)
                if c["causal"]:
                    at = torch.arange(a, b, device=DEV) - starts[i + 1] + n
                    at = at.repeat_interleave(G)[:, None]
                    key = torch.arange(n, device=DEV)[None]
                    hide = key > at
                    if c["window"]:
                        hide |= key <= at - c["window"]
                    score[hide] = -math.inf
                out[a:b, h * G:(h + 1) * G] = torch.mm(torch.softmax(score, 1), v).view(b - a, G, D)
    return out
