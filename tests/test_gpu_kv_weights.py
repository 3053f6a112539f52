"""Attention over the paged 8-bit cache where one key holds most of a row's
weight and a long tail shares the rest (the first token of a text, in language
models): the tail's small weights have to be there.  The bound counts a weight's
rounding within its own tile of 64 tokens, so it does not grow with the context."""
import numpy as np
import pytest

from .gpu_common import require_gpu, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
QTOP = {"f32": 8355711.0, "bf16": 32639.0}     # integers of a query row, by output type
PTOP = 8355711.0                               # integers of a tile's largest weight
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # half a step of a rounded output, relative


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def definition(q, k, v, scale, out, many):
    """Rows q [n][D] that see all of k, v [L][D] (64 bits, on the GPU): the output
    and how far the library's may be off.

    Few columns:
    - A score is off by scale sum |k| times half an integer step of the query
      and two fp32 roundings, and relatively by its own: factor 6, joined digits
      2; the subtractions of the tile's maximum, of the wave's from the tile's
      and of the row's from the wave's and the workgroup's round relative to
      differences of scores, at most twice the largest: 8 + 4 * 2 < 24.
    - A weight is exp2 of the score less its tile's maximum times exp2 of that
      one less the running maximum: 2 u each, 2 u more for the products.
    - On top of that a weight is rounded to integers of 1 / PTOP of its tile's
      largest, once, so by half of one.
    - The sums: 16 terms in a lane, 2 levels across lanes, then a product, a sum
      and a rescaling (4 u) for each of a wave's tiles (a quarter of the
      workgroup's; or fewer, and as many shares), 4 waves, the scales and the
      quotient: (tiles + 60) u.
    The quotient takes both sums' errors.
    Many columns: a query's channel and a weight are off relatively by c = 2^-12
    (fp32: 2^-23, in two parts), a weight by no less than steps of 2^-31 (2^-38) of
    the row's largest; a sum of D products is off by D u of its terms' sizes, one of
    L weights by L u."""
    import torch
    L = k.shape[0]
    s = scale * (q @ k.t().contiguous())
    e = torch.exp(s - s.amax(1, keepdim=True))
    total = e.sum(1, keepdim=True)
    w = e / total
    o, V = w @ v, w @ v.abs()
    A = abs(scale) * q.abs().amax(1) * k.abs().sum(1).max()
    ds = A * (0.5 / QTOP[out] + 2 * U) + 24 * U * s.abs().amax(1)
    tiles = -(-L // 64)
    pad = torch.nn.functional.pad
    most = pad(w, (0, 64 * tiles - L)).view(-1, tiles, 64).amax(2)                   # [n][tiles]
    size = pad(v.abs(), (0, 0, 0, 64 * tiles - L)).view(tiles, 64, -1).sum(1)        # [tiles][D]
    grid = 0.5 / PTOP * (most @ size)
    rel = ds[:, None] + (6 + tiles + 60) * U
    if many:
        c = 2.0 ** -12 if out == "bf16" else 2.0 ** -23
        sizes = abs(scale) * (q.abs() @ k.abs().t().contiguous()).amax(1)
        rel = (sizes * (c + q.shape[1] * U) + 24 * U * s.abs().amax(1))[:, None] + c + (L + tiles + 100) * U
        grid = L * 2.0 ** (-31 if out == "bf16" else -38) * w.amax(1, keepdim=True) * v.abs().amax(0)
    return o, 1.05 * (2 * rel * V + grid) + HALF[out] * o.abs() + 1e-37


# sequences, their length, key heads, group, channels, tokens of a page
FORMS = [
    (64, 2048, 4, 2, 64, 64),       # sequences whole, a workgroup each
    (64, 4096, 4, 1, 128, 128),
    (1, 4096, 2, 8, 128, 64),       # dealt out
    (40, 8192, 8, 4, 64, 64),       # dealt out, long runs
    (2, 32768, 1, 4, 256, 256),
    (1, 32768, 2, 3, 64, 64),
    (1025, 32768, 1, 2, 64, 64),    # more sequences than are dealt out: one of that length, the others of one token
    (1025, 8192, 1, 2, 128, 64),
]


@pytest.mark.parametrize("S,L,Hkv,G,D,page", FORMS)
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("tail", [("share", 0.9), ("share", 0.97), ("flat", 11.2), ("flat", 14.0), ("flat", 16.8)])
def test_small_weights_beside_a_large_one(S, L, Hkv, G, D, page, out, many, tail):
    """share: the first key holds that share of the weight and its value is near
    0, the others' scores are normal (0.3).  flat: the others lie that many nats
    below, all values are of one sign."""
    import moe_decode_amd as md
    import torch
    say(f"[weights] {S} x {L} {Hkv} {G} {D} {page} {out} {many} {tail}")
    kind, much = tail
    rng = np.random.default_rng(L + D)
    n = -(-L // page)
    shape = (n, Hkv, page, D)
    k = np.rint(6 * rng.standard_normal(shape)) if kind == "share" else np.zeros(shape)
    k[..., 0] = 0
    v = rng.integers(32, 97, shape)
    perm = rng.permutation(n)
    k[perm[0], :, 0] = 0
    k[perm[0], :, 0, 0] = 127
    if kind == "share":
        v[perm[0], :, 0] = rng.integers(-1, 2, (Hkv, D))
    ks, vs, scale = np.float32(0.05), np.float32(0.02), D ** -0.5

    def gpu(a, t=torch.int8):
        return torch.from_numpy(a).to("cuda", t).contiguous()
    kg, vg = gpu(k), gpu(v)
    c = md.KVCache(kg, vg.transpose(2, 3).contiguous(), torch.full((n, Hkv), float(ks), device="cuda"),
                   torch.full((n, Hkv), float(vs), device="cuda"))
    order = torch.from_numpy(perm).cuda()
    kd = (kg[order].double() * float(ks)).transpose(0, 1).reshape(Hkv, n * page, D)[:, :L]
    vd = (vg[order].double() * float(vs)).transpose(0, 1).reshape(Hkv, n * page, D)[:, :L]
    rows = min(S, 64)
    q = torch.from_numpy(rng.standard_normal((S, Hkv * G, D))).cuda()
    q[..., 0] = 0
    for h in range(Hkv):        # the first channel reaches the first key alone and makes its score
        for g in range(G):
            x = q[:rows, h * G + g]
            if kind == "share":
                s = scale * (x @ kd[h, 1:].t().contiguous())
                s0 = torch.logsumexp(s, 1) + float(np.log(much / (1 - much)))
            else:
                s0 = much
            q[:rows, h * G + g, 0] = s0 / (scale * 127 * float(ks))
    q = q.float()
    lens, table = [L] * S, np.tile(perm, (S, 1))        # (all sequences on the same pages)
    if S > 1024:
        lens = [1] * S
        lens[3], rows = L, 4
        q[3] = q[0]
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")  # noqa: E731
    b = md.KVBatch(i32(range(S + 1)), i32(lens), i32(table), 800 if many else 1, L)
    got = md.kv_attention(c, b, q, scale=scale, out_dtype={"f32": torch.float32, "bf16": torch.bfloat16}[out]).double()
    seen = [3] if S > 1024 else list(range(rows))
    worst, off, wide = 0.0, 0.0, 0.0
    for h in range(Hkv):
        for g in range(G):
            want, tol = definition(q[seen, h * G + g].double(), kd[h], vd[h], scale, out, many)
            err = (got[seen, h * G + g] - want).abs()
            worst = max(worst, float((err / tol).max()))
            off = max(off, float((err.norm(dim=1) / want.norm(dim=1)).max()))
            wide = max(wide, float((tol.norm(dim=1) / want.norm(dim=1)).max()))
    say(f"  error / bound {worst:.3f}, relative {off:.2e}, the bound {wide:.2e}")
    assert wide <= (0.02 if out == "bf16" or many else 1e-3)       # (the bound says something)
    assert worst <= 1.0, (worst, off)
    if S > 1024:    # the sequences of one token: its value, of a weight that is off by half of 1 / PTOP and a few u
        one = [s for s in range(S) if s != 3]
        first = vd[:, :1].expand(-1, G, -1).reshape(Hkv * G, D)
        assert bool(((got[one] - first).abs() <= (HALF[out] + (2.0 ** -12 if many and out == "bf16" else 16 * U)) * first.abs()).all())
