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
