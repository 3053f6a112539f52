"""Routing on the GPU: the experts are the definition's, from logits in 64 bits
rounded once; gates within the rounding of their last step."""
import numpy as np
import pytest

from . import step_model as M
from .gpu_common import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _inputs(rng, T, H, E, xt):
    import torch
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32))
    x = x.to({"f32": torch.float32, "bf16": torch.bfloat16}[xt])
    W = (1.5 / np.sqrt(H) * rng.standard_normal((E, H))).astype(np.float32)
    return x.cuda(), torch.from_numpy(W).cuda(), x.float().numpy().astype(np.float64) @ W.astype(np.float64).T


def _check(x, W, exact, k, score="softmax", balance=None, groups=1, kept=1, best_two=False, renorm=True, scale=1.0,
           bias=None):
    import moe_decode_amd as md
    import torch
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    r = md.Routing(k, score, dev(balance), groups, kept, best_two, renorm, scale)
    T, E = exact.shape
    logits = torch.empty(T, E, device="cuda")
    idx, gates = md.moe_route(x, W, r, bias=dev(bias), logits=logits)
    l = (exact if bias is None else exact + bias.astype(np.float64)).astype(np.float32)
    got = logits.cpu().numpy()
    # the sum's last bits may fall on the other side of a tie of fp32: one step
    assert (np.abs(got - l) <= np.spacing(np.abs(l))).all() and (got != l).mean() < 1e-4
    idx, gates = idx.cpu().numpy(), gates.cpu().numpy()
    for t in range(T):
        won, g = M.route(got[t], k, score, balance, groups, kept, best_two, renorm, scale)
        assert idx[t].tolist() == won, (t, idx[t].tolist(), won)
        assert (np.abs(gates[t] - g) <= M.U * np.abs(g) * 1.001 + 1e-45).all(), (t, gates[t], g)


OPTIONS = [dict(), dict(score="sigmoid"), dict(score="sigmoid", balance=0.1, groups=4, kept=2, best_two=True, scale=2.5),
           dict(balance=0.02, renorm=False), dict(groups=2, kept=1), dict(score="sigmoid", groups=4, kept=3, renorm=False),
           dict(groups=4, kept=4, best_two=True), dict(score="sigmoid", bias=1.0, balance=0.05)]


@pytest.mark.parametrize("T,H,E", [(1, 256, 8), (1, 2048, 128), (3, 6144, 256), (8, 512, 60), (9, 512, 60), (17, 2048, 128),
                                   (128, 6144, 256), (65, 768, 4), (300, 256, 160), (1000, 512, 64)])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_sizes_and_options(T, H, E, xt):
    rng = np.random.default_rng(T + E)
    x, W, exact = _inputs(rng, T, H, E, xt)
    for o in OPTIONS:
        o = dict(o)
        for name in ("balance", "bias"):
            if name in o:
                o[name] = (o[name] * rng.standard_normal(E)).astype(np.float32)
        n = E // o.get("groups", 1)
        if o.get("best_two") and n < 2:
            continue
        _check(x, W, exact, min(8, n * o.get("kept", 1)), **o)
    _check(x, W, exact, 1)


@pytest.mark.parametrize("E,groups,kept", [(64, 64, 8), (256, 64, 7), (96, 3, 2), (160, 5, 4), (120, 40, 3), (6, 2, 1),
                                           (2, 1, 1)])
def test_group_shapes(E, groups, kept):
    rng = np.random.default_rng(E)
    for T in (2, 40):
        x, W, exact = _inputs(rng, T, 512, E, "f32")
        k = min(8, kept * (E // groups))
        _check(x, W, exact, k, "sigmoid", (0.1 * rng.standard_normal(E)).astype(np.float32), groups, kept)
        if E // groups > 1:
            _check(x, W, exact, k, "softmax", None, groups, kept, True)


@pytest.mark.parametrize("T", [2, 50])
def test_equal_scores_go_to_the_lower_run_and_expert(T):
    """Experts with the same row of weights, and a row of zeros."""
    import torch
    rng = np.random.default_rng(T)
    x, W, exact = _inputs(rng, T, 256, 64, "f32")
    W[32:] = W[:32]
    exact[:, 32:] = exact[:, :32]
    x[1] = 0.0
    exact[1] = 0.0
    for score in ("softmax", "sigmoid"):
        _check(x, W, exact, 8, score)
        _check(x, W, exact, 8, score, None, 8, 3)
        _check(x, W, exact, 8, score, None, 8, 3, True)
        _check(x, W, exact, 6, score, np.tile(np.float32([0.25, 0.5]), 32), 4, 2)


@pytest.mark.parametrize("T", [2, 50])
def test_far_logits_and_closed_experts(T):
    """Logits past exp's range, experts closed by a balance of -inf."""
    rng = np.random.default_rng(T)
    x, W, exact = _inputs(rng, T, 256, 32, "f32")
    bias = np.zeros(32, np.float32)
    bias[3], bias[9] = 900.0, -900.0
    _check(x, W, exact, 3, "softmax", bias=bias)
    _check(x, W, exact, 8, "sigmoid", bias=bias)
    shut = np.zeros(32, np.float32)
    shut[5:] = -np.inf
    _check(x, W, exact, 8, "sigmoid", shut)
    _check(x, W, exact, 4, "softmax", shut, 4, 2)


@pytest.mark.parametrize("T", [3, 70])
def test_a_nan_keeps_to_its_token(T):
    import moe_decode_amd as md
    import torch
    rng = np.random.default_rng(T)
    x, W, _ = _inputs(rng, T, 512, 60, "f32")
    r = md.Routing(6, "sigmoid", groups=4, groups_kept=2)
    idx, gates = md.moe_route(x, W, r)
    x[1, 7] = float("nan")
    idx2, gates2 = md.moe_route(x, W, r)
    keep = torch.arange(T, device="cuda") != 1
    assert torch.equal(idx[keep], idx2[keep]) and torch.equal(gates[keep], gates2[keep])
    got = idx2[1].tolist()
    assert len(set(got)) == 6 and all(0 <= e < 60 for e in got)


def test_rows_behind_and_captured_calls():
    import moe_decode_amd as md
    import torch
    rng = np.random.default_rng(4)
    for T in (5, 200):
        x, W, _ = _inputs(rng, T, 512, 128, "bf16")
        r = md.Routing(8, "sigmoid", torch.rand(128, device="cuda"), 8, 4, True, scale=2.0)
        idx = torch.full((T + 1, 8), -3, dtype=torch.int32, device="cuda")
        gates = torch.full((T + 1, 8), -3.0, device="cuda")
        md.moe_route(x, W, r, idx=idx[:T], gates=gates[:T])
        assert (idx[T] == -3).all() and (gates[T] == -3.0).all()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gi, gg = md.moe_route(x, W, r)
        for i in range(3):
            x.copy_(torch.randn(T, 512, device="cuda"))
            graph.replay()
            torch.cuda.synchronize()
            ei, eg = md.moe_route(x, W, r)
            assert torch.equal(gi, ei) and torch.equal(gg, eg)
    i0, g0 = md.moe_route(x[:0], W, r)
    assert i0.shape == (0, 8) and g0.shape == (0, 8)


@pytest.mark.parametrize("T", [1, 5, 33])
def test_the_layer_with_a_routing(T):
    """moe_layer_forward(routing=...) is moe_route and moe_experts_forward; a softmax
    over the chosen ones is the layer's own routing."""
    import moe_decode_amd as md
    import torch

    from .gpu_common import moe_layer
    layer = moe_layer("c3")
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, layer.H, generator=g, device="cuda")
    r = md.Routing(layer.k, "sigmoid", 0.05 * torch.randn(layer.E, generator=g, device="cuda"), 8, 4, True, scale=2.5)
    idx, gates = md.moe_route(x, layer.Wr, r, bias=layer.bias)
    want = md.moe_experts_forward(layer, x, idx, gates)
    i2, g2 = torch.empty_like(idx), torch.empty_like(gates)
    y = md.moe_layer_forward(layer, x, idx=i2, gates=g2, routing=r)
    assert torch.equal(y, want) and torch.equal(i2, idx) and torch.equal(g2, gates)
    assert torch.equal(md.moe_layer_forward(layer, x, routing=r), want)
    i3, g3 = torch.empty_like(idx), torch.empty_like(gates)
    md.moe_layer_forward(layer, x, idx=i3, gates=g3)
    i4, g4 = md.moe_route(x, layer.Wr, md.Routing(layer.k), bias=layer.bias)
    assert torch.equal(i3, i4) and (g3 - g4).abs().max() <= 2.0 ** -23


# ---- many tokens: logits bounded first ---------------------------------------

def _off(x, W):
    """How far the bounded form's logits may be off: 2^-19 |x| |w|, and one step of
    fp32 that the definition's rounding has."""
    l = x.double() @ W.double().t()
    n = x.double().norm(dim=1, keepdim=True) * W.double().norm(dim=1).max()
    return (2.0 ** -19 * n + 2.0 ** -23 * l.abs().amax(1, keepdim=True)).cpu().numpy()


MANY = [(2100, 4096, 256, "f32"), (8191, 1024, 256, "bf16"), (9001, 2304, 100, "f32"), (1100, 8192, 256, "bf16"),
        (4000, 6144, 129, "bf16"), (19001, 2304, 100, "f32"), (1023, 6144, 256, "bf16")]


@pytest.mark.parametrize("T,H,E,xt", MANY)
@pytest.mark.parametrize("kind", ["random", "close", "same", "positive"])
def test_many_tokens_choose_as_few(T, H, E, xt, kind):
    """The experts are those of the form that keeps every logit in fp64 (a call that
    asks for the logits); a gate is off by what its logit's bound allows.  `close`:
    experts that differ in the last bits of their weights, `same`: pairs of equal
    ones, `positive`: sums without any cancellation."""
    import moe_decode_amd as md
    import torch
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, H, generator=g, device="cuda")
    W = torch.randn(E, H, generator=g, device="cuda") * (1.5 / H ** 0.5)
    if kind == "positive":
        x, W = x.abs(), W.abs() / H ** 0.5
    if kind in ("close", "same"):
        W[E // 2:] = W[:E - E // 2] * (1 + 2.0 ** -22 if kind == "close" else 1)
    x = x.to({"f32": torch.float32, "bf16": torch.bfloat16}[xt])
    logits = torch.empty(T, E, device="cuda")
    off = _off(x, W)
    for r in (md.Routing(8, "sigmoid", 0.05 * torch.randn(E, generator=g, device="cuda"), scale=2.5),
              md.Routing(6, renorm=False), md.Routing(3, "softmax", 0.5 / E * torch.randn(E, generator=g, device="cuda")),
              md.Routing(4, "sigmoid", groups=2 if E % 2 == 0 else 1, best_two=True)):
        idx, gates = md.moe_route(x, W, r)
        want, wg = md.moe_route(x, W, r, logits=logits)
        assert torch.equal(idx, want), (idx != want).any(1).nonzero()[:4].tolist()
        # a score moves by the factor exp(2 off) at most, a sum of them too
        err, wg = (gates - wg).abs().cpu().numpy(), wg.abs().cpu().numpy()
        assert (err <= wg * (4.1 * off + 4 * M.U)).all(), float((err / wg).max())


@pytest.mark.parametrize("T,H,E,xt", [(2999, 6144, 256, "bf16"), (2999, 6144, 200, "f32"), (5001, 4096, 100, "bf16")])
def test_many_tokens_of_uneven_columns(T, H, E, xt):
    """Values whose sizes differ by orders of magnitude: from column to column, from
    one run of 64 columns to the next (x one way, W_r the other) and from token to
    token; and one column alone."""
    import moe_decode_amd as md
    import torch
    g = torch.Generator(device="cuda").manual_seed(T + E)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    runs = torch.exp2(torch.randint(-30, 31, (H // 64,), generator=g, device="cuda").float()).repeat_interleave(64)
    x, W = rn(T, H), rn(E, H) * (1.5 / H ** 0.5)
    alone = torch.zeros(H, device="cuda")
    alone[H // 2 + 5] = H ** 0.5
    cases = [(x * torch.exp(2 * rn(T, H)) / 8, W * torch.exp(2 * rn(E, H)) / 8), (x * runs, W / runs),
             (x * torch.exp2(torch.randint(-8, 3, (T, 1), generator=g, device="cuda").float()), W), (x * alone, W)]
    logits = torch.empty(T, E, device="cuda")
    for x, W in cases:
        x = x.to({"f32": torch.float32, "bf16": torch.bfloat16}[xt])
        off = _off(x, W)
        for r in (md.Routing(8, "sigmoid", 0.05 * rn(E), scale=2.5), md.Routing(6, renorm=False)):
            idx, gates = md.moe_route(x, W, r)
            want, wg = md.moe_route(x, W, r, logits=logits)
            assert torch.equal(idx, want), (idx != want).any(1).nonzero()[:4].tolist()
            err, wg = (gates - wg).abs().cpu().numpy(), wg.abs().cpu().numpy()
            # where the bound is above 0.01 every token is done in fp64
            assert (err <= wg * (4.1 * np.minimum(off, 0.01) + 4 * M.U)).all(), float((err / wg).max())


def test_many_tokens_special_values():
    """Zeros (all experts equal), NaN and infinities in some tokens, closed experts,
    weights near the smallest normal numbers."""
    import moe_decode_amd as md
    import torch
    T, H, E = 2100, 4096, 256
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(T, H, generator=g, device="cuda")
    W = torch.randn(E, H, generator=g, device="cuda") * (1.5 / H ** 0.5)
    logits = torch.empty(T, E, device="cuda")
    shut = torch.zeros(E, device="cuda")
    shut[10:] = float("-inf")
    x[3], x[7, 9], x[8, 1], x[2099, 0] = 0.0, float("nan"), float("inf"), 3e38
    x[64:128] *= 1e-30
    for w in (W, torch.zeros_like(W), W * 1e-37):
        for r in (md.Routing(8, "sigmoid"), md.Routing(8, "sigmoid", shut), md.Routing(2, "softmax", None, 8, 3)):
            idx, gates = md.moe_route(x, w, r)
            want, wg = md.moe_route(x, w, r, logits=logits)
            keep = torch.isfinite(x).all(1)
            assert torch.equal(idx[keep], want[keep])
            ok = torch.isclose(gates, wg, rtol=1e-3, atol=0, equal_nan=True)
            assert ok[keep].all()
            assert ((idx >= 0) & (idx < E)).all() and (idx.sort(1).values.diff(dim=1) > 0).all()


def test_many_tokens_captured():
    import moe_decode_amd as md
    import torch
    T, H, E = 2100, 4096, 256
    x = torch.randn(T, H, device="cuda").bfloat16()
    W = torch.randn(E, H, device="cuda") * (1.5 / H ** 0.5)
    r = md.Routing(8, "sigmoid", None, 8, 4, True)
    graph = torch.cuda.CUDAGraph()
    md.moe_route(x, W, r)
    with torch.cuda.graph(graph):
        gi, gg = md.moe_route(x, W, r)
    for i in range(3):
        x.copy_(torch.randn(T, H, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        ei, eg = md.moe_route(x, W, r)
        assert torch.equal(gi, ei) and torch.equal(gg, eg)
