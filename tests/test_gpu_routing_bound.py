"""Routing of many tokens on the GPU, where logits are bounded first and only the
tokens that the bound leaves open are done in fp64: which tokens those are, and the
bound itself."""
import pytest

from .gpu_common import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _problem(T, H, E, xt, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, generator=g, device="cuda").to({"f32": torch.float32, "bf16": torch.bfloat16}[xt])
    return g, x, torch.randn(E, H, generator=g, device="cuda") * (1.5 / H ** 0.5)


@pytest.mark.parametrize("options", [dict(score="sigmoid"), dict(score="sigmoid", groups=8, groups_kept=4, best_two=True),
                                     dict(score="softmax"), dict(score="softmax", groups=8, groups_kept=3)])
@pytest.mark.parametrize("far", [-1e9, -3.4028234663852886e38])
def test_experts_closed_by_a_finite_balance_leave_the_others_alone(options, far):
    """The same bits as with -inf, so the same tokens are done in fp64: a margin that
    the far expert's size sets would leave all of them open, and their gates would be
    fp64's, which differ in some last places."""
    import moe_decode_amd as md
    import torch
    T, H, E = 4001, 6144, 256
    g, x, W = _problem(T, H, E, "bf16", 5)
    scale = 0.05 if options["score"] == "sigmoid" else 0.5 / E
    balance = scale * torch.randn(E, generator=g, device="cuda")
    got = {}
    for value in (far, float("-inf")):
        b = balance.clone()
        b[[3, 17, 200]] = value
        got[value] = md.moe_route(x, W, md.Routing(8, balance=b, **options))
    logits = torch.empty(T, E, device="cuda")
    want, wg = md.moe_route(x, W, md.Routing(8, balance=b, **options), logits=logits)
    for idx, gates in got.values():
        assert torch.equal(idx, want)
    (_, a), (_, b) = got.values()
    assert torch.equal(a, b)
    assert not torch.equal(b, wg)       # else this test sees nothing


# ---- the bound ---------------------------------------------------------------

UNITS = {"bf16": 6.25, "f32": 9.25}     # of 2^-23 |x| |w|, as documented
U = 2.0 ** -24


def _bound(x, W, l):
    """Of each token: what a logit may be off by, and half a step of fp32 for the
    definition's rounding (twice that: l may be a little larger there)."""
    import torch
    n = x.double().norm(dim=1, keepdim=True) * W.double().norm(dim=1).max()
    return UNITS["f32" if x.dtype == torch.float32 else "bf16"] * 2.0 ** -23 * n + 2 * U * l.abs().amax(1, keepdim=True)


def _uneven(g, x, W, kind):
    import torch
    T, H = x.shape
    if kind == "positive":              # sums without any cancellation
        return x.abs(), W.abs() / H ** 0.5
    if kind == "columns":               # sizes over orders of magnitude, few products make the sum
        a = torch.exp(2 * torch.randn(T, H, generator=g, device="cuda")) / 8
        b = torch.exp(2 * torch.randn(W.shape, generator=g, device="cuda")) / 8
        x, W = (x.float() * a).to(x.dtype), W * b
        return x, W * (100 / (x.double().norm(dim=1).mean() * W.double().norm(dim=1).max()).float())
    if kind == "runs":                  # from one run of 64 columns to the next, x one way and W the other
        r = torch.exp2(torch.randint(-30, 31, (H // 64,), generator=g, device="cuda").float()).repeat_interleave(64)
        x, W = (x.float() * r).to(x.dtype), W / r
        return x, W * (100 / (x.double().norm(dim=1).mean() * W.double().norm(dim=1).max()).float())
    return x, W


@pytest.mark.parametrize("T,H,E,xt", [(8191, 6144, 256, "bf16"), (8191, 2048, 128, "f32"), (3001, 6144, 200, "f32"),
                                      (8191, 4096, 60, "bf16"), (2100, 16384, 256, "bf16")])
@pytest.mark.parametrize("kind", ["random", "positive", "columns", "runs"])
def test_logits_are_within_the_documented_bound(T, H, E, xt, kind):
    """A gate by sigmoid, not renormalised, is its logit's: a large balance names the
    experts, and l = log(g / (1 - g)), where half a step of the gate moves l by u / (1 - g)."""
    import moe_decode_amd as md
    import torch
    g, x, W = _problem(T, H, E, xt, T + H)
    x, W = _uneven(g, x, W, kind)
    l = x.double() @ W.double().t()
    bound, far = _bound(x, W, l), 0.0
    for first in range(0, E, max(8, E // 40 * 8)):
        balance = torch.zeros(E, device="cuda")
        balance[first:first + 8] = 16.0
        idx, gates = md.moe_route(x, W, md.Routing(min(8, E - first), "sigmoid", balance, renorm=False))
        assert ((idx >= first) & (idx < first + 8)).all()
        p = gates.double()
        got, want = torch.log(p / (1 - p)), l.gather(1, idx.long())
        ok = (p > 0) & (p < 1)
        tol = bound + 1.05 * U / (1 - p)
        err = (got - want).abs()
        assert (err <= tol)[ok].all(), float((err / tol)[ok].max())
        assert ok.double().mean() > 0.9
        far = max(far, float((err / bound)[ok & (p < 0.9)].max()))
    print(f"{T} x {H} x {E} {xt} {kind}: {far:.3f} of the bound")


CALLS = [dict(k=8, score="sigmoid", groups=8, groups_kept=4, best_two=True, scale=2.5, balance=0.05, bias=0.3),
         dict(k=8, score="softmax", groups=8, groups_kept=4, best_two=True, scale=2.5, balance=0.002, bias=0.3),
         dict(k=5, score="sigmoid", groups=5, groups_kept=2, balance=0.05), dict(k=6, groups=5, groups_kept=3, balance=0.002),
         dict(k=3, score="sigmoid", groups=4, groups_kept=1, renorm=False, bias=2.0), dict(k=8, bias=1.0, renorm=False),
         dict(k=2, score="sigmoid", groups=20, groups_kept=7, best_two=True, balance=0.2), dict(k=1, score="sigmoid")]


def _calls(E, g):
    """The options that divide E, as Routing and bias."""
    import moe_decode_amd as md
    import torch
    for o in CALLS:
        o = dict(o)
        if E % o.get("groups", 1):
            continue
        rn = lambda s: s * torch.randn(E, generator=g, device="cuda")  # noqa: E731
        b, bias = o.pop("balance", None), o.pop("bias", None)
        yield md.Routing(o.pop("k"), balance=None if b is None else rn(b), **o), None if bias is None else rn(bias)


MANY = [(8191, 4096, 60, "bf16"), (8191, 4096, 60, "f32"), (8191, 4096, 64, "f32"), (4001, 4096, 160, "bf16"),
        (4001, 4096, 160, "f32"), (3001, 6144, 256, "bf16"), (2101, 6144, 256, "f32"), (5003, 2304, 200, "bf16"),
        (8191, 2048, 128, "bf16")]


@pytest.mark.parametrize("T,H,E,xt", MANY)
@pytest.mark.parametrize("kind", ["random", "close"])
def test_options_of_many_tokens(T, H, E, xt, kind):
    """The experts of the form that keeps every logit in fp64, and gates that are off
    by what the documented bound allows: a score moves by the factor exp(2 off) at most,
    a sum of them too."""
    import moe_decode_amd as md
    import torch
    g, x, W = _problem(T, H, E, xt, T + E)
    if kind == "close":
        W[E // 2:] = W[:E - E // 2] * (1 + 2.0 ** -22)
    logits = torch.empty(T, E, device="cuda")
    for r, bias in _calls(E, g):
        l = x.double() @ W.double().t() + (0.0 if bias is None else bias.double())
        idx, gates = md.moe_route(x, W, r, bias=bias)
        want, wg = md.moe_route(x, W, r, bias=bias, logits=logits)
        assert torch.equal(idx, want), (vars(r), (idx != want).any(1).nonzero()[:4].tolist())
        err = (gates - wg).abs().double()
        assert (err <= wg.abs() * (4.1 * _bound(x, W, l) + 4 * U)).all(), (vars(r), float((err / wg).max()))


def test_options_captured():
    """Replays against the form that keeps every logit in fp64."""
    import moe_decode_amd as md
    import torch
    T, H, E = 2101, 6144, 256
    g, x, W = _problem(T, H, E, "bf16", 9)
    logits = torch.empty(T, E, device="cuda")
    for r, bias in list(_calls(E, g))[:2]:
        md.moe_route(x, W, r, bias=bias)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gi, gg = md.moe_route(x, W, r, bias=bias)
        for _ in range(3):
            x.copy_(torch.randn(T, H, generator=g, device="cuda"))
            graph.replay()
            torch.cuda.synchronize()
            want, wg = md.moe_route(x, W, r, bias=bias, logits=logits)
            assert torch.equal(gi, want)
            l = x.double() @ W.double().t() + bias.double()
            assert ((gg - wg).abs().double() <= wg.abs() * (4.1 * _bound(x, W, l) + 4 * U)).all()


@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("options", [dict(score="sigmoid"), dict(renorm=False)])
def test_a_bound_above_2_to_minus_10_takes_fp64(xt, options):
    """A large value of x that W_r does not see leaves the logits as they are and makes
    their bound one that would allow gates 0.8% off: they are fp64's, to the bit."""
    import moe_decode_amd as md
    import torch
    T, H, E = 3001, 6144, 256
    g, x, W = _problem(T, H, E, xt, 31)
    x[:, 70], W[:, 70] = 2000.0, 0.0
    off = _bound(x, W, x.double() @ W.double().t())
    assert 2.0 ** -10 < off.min() and off.max() < 2.0 ** -8
    r = md.Routing(8, **options)
    idx, gates = md.moe_route(x, W, r)
    want, wg = md.moe_route(x, W, r, logits=torch.empty(T, E, device="cuda"))
    assert torch.equal(idx, want) and torch.equal(gates, wg)
