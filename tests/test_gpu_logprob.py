"""Log probabilities, entropy and alternatives on the GPU: ids equal to the order
of the definition, values within the bound derived in step_model.py."""
import numpy as np
import pytest

from . import step_model as M
from .gpu_common import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _logits(rng, rows, V, xt, stride=0, offset=0):
    """A view [rows][V] with the given row stride that begins `offset` values in."""
    import torch
    x = 2 * rng.standard_normal((rows, V))
    x[np.arange(rows), rng.integers(0, V, rows)] += 9
    t = torch.from_numpy(x.astype(np.float32)).to({"f32": torch.float32, "bf16": torch.bfloat16}[xt])
    stride = stride or V
    flat = torch.full((offset + rows * stride + 16,), 1e30, dtype=t.dtype, device="cuda")     # around: never read as logits
    view = flat[offset:offset + rows * stride].view(rows, stride)[:, :V]
    view.copy_(t)
    return view


def _check(x, tokens, top, scale, ids=True):
    import moe_decode_amd as md
    import torch
    a = x.float().cpu().numpy()
    r = md.token_logprobs(x, None if tokens is None else torch.from_numpy(tokens).cuda(), top, scale)
    lp, tol, H, htol = M.logprobs(a, float(np.float32(scale)))
    got = r.entropy.cpu().numpy()
    assert (np.abs(got - H) <= htol).all(), float((np.abs(got - H) / htol).max())
    rows = np.arange(len(a))[:, None]

    def near(g, at):
        w, t = lp[rows, at], tol[rows, at]
        # the type's lowest value times 1.3 is -4.4e38: past the largest fp32 (3.4028e38), rounded to -inf
        w = np.where(w < -(2.0 ** 128 - 2.0 ** 103), -np.inf, w)
        ok = np.where(np.isfinite(w), np.abs(g - w) <= t, g == w)
        assert ok.all(), (np.argwhere(~ok)[:4].tolist(), g[~ok][:4], w[~ok][:4])
    if tokens is None:
        assert r.logprobs is None
    else:
        near(r.logprobs.cpu().numpy(), tokens)
    if top:
        want = M.top_ids(a, top)
        got = r.top_ids.cpu().numpy()
        assert np.array_equal(got, want), np.argwhere(got != want)[:4].tolist()
        near(r.top_logprobs.cpu().numpy(), want)
    else:
        assert r.top_ids is None and r.top_logprobs is None


SHAPES = [(1, 1), (1, 2), (3, 7), (5, 100), (1, 2041), (2, 2048), (2, 2049), (9, 8185), (4, 8193), (1, 32000), (7, 32003),
          (2, 131071), (600, 513), (520, 8200), (1, 1 << 20), (2, 300001)]


@pytest.mark.parametrize("rows,V", SHAPES)
@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_sizes(rows, V, xt):
    rng = np.random.default_rng(rows + V)
    x = _logits(rng, rows, V, xt)
    for top, n, scale in [(0, 1, 1.0), (min(V, 5), 3, 0.7), (min(V, 32), 0, 1.9)]:
        tokens = rng.integers(0, V, (rows, n)).astype(np.int32) if n else None
        _check(x, tokens, top, scale)


@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("offset", range(9))
def test_rows_that_begin_anywhere(xt, offset):
    rng = np.random.default_rng(offset)
    for V, stride in ((101, 0), (2045, 2051), (8187, 8191), (4099, 5000)):
        x = _logits(rng, 3, V, xt, stride, offset)
        _check(x, rng.integers(0, V, (3, 2)).astype(np.int32), 4, 1.0)


@pytest.mark.parametrize("V", [40, 2048, 5000, 40000])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_equal_logits_go_to_the_lower_id(V, xt):
    import torch
    rng = np.random.default_rng(V)
    x = _logits(rng, 6, V, xt)
    x[0] = 1.5                                                # all equal
    x[1] = x[1].round()                                       # many equal ones
    x[2] = torch.arange(V, device="cuda").float() / V         # ascending
    x[3] = -torch.arange(V, device="cuda").float() / V
    x[4] = 0.0
    x[4, ::2] = -0.0                                          # one value
    for top in (1, 20, 32):
        _check(x, None, top, 1.0)


@pytest.mark.parametrize("V", [50, 3000, 70000])
def test_masked_logits(V):
    """-inf in most places; a row of one token; rows with fewer tokens left than asked for."""
    import torch
    rng = np.random.default_rng(V)
    x = _logits(rng, 5, V, "f32")
    x[0, torch.from_numpy(rng.permutation(V)[: V - 30]).cuda()] = float("-inf")
    x[1] = float("-inf")
    x[1, V - 1] = -3.0e38
    x[2, : V // 2] = float("-inf")
    x[3, 1:] = torch.finfo(torch.float32).min                 # the type's lowest value, and one token
    x[4, V // 3:] = float("-inf")
    _check(x, rng.integers(0, V, (5, 6)).astype(np.int32), 32, 1.0)
    tok = np.tile(np.array([0, V - 1], np.int32), (5, 1))
    _check(x, tok, 1, 1.3)


@pytest.mark.parametrize("V", [50, 3000, 70000])
def test_rows_that_have_no_distribution(V):
    """NaN, +inf, nothing but -inf: NaN in all values of the row, the others as
    they were, ids still the order's; a token that is none gives NaN."""
    import moe_decode_amd as md
    import torch
    rng = np.random.default_rng(V)
    x = _logits(rng, 6, V, "f32")
    x[1, V // 2] = float("nan")
    x[2, 3] = float("inf")
    x[3] = float("-inf")
    x[4] = float("nan")
    tok = np.tile(np.array([[3, V // 2]], np.int32), (6, 1))
    tok[5] = [-1, V]
    r = md.token_logprobs(x, torch.from_numpy(tok).cuda(), 8)
    for row in (1, 2, 3, 4):
        assert r.entropy[row].isnan() and r.logprobs[row].isnan().all() and r.top_logprobs[row].isnan().all()
    assert np.array_equal(r.top_ids.cpu().numpy(), M.top_ids(x.cpu().numpy(), 8))
    assert r.logprobs[5].isnan().all() and not r.entropy[5].isnan()
    good = md.token_logprobs(x[:1], torch.from_numpy(tok[:1]).cuda(), 8)
    for a, b in zip(r, good):
        assert torch.equal(a[:1], b)


@pytest.mark.parametrize("V", [16384, 16385, 24001, 32761, 32762])
def test_rows_of_one_step(V):
    """Around the lengths that one workgroup takes in one step: each of the cases above."""
    rng = np.random.default_rng(V)
    for xt in ("f32", "bf16"):
        test_sizes(1, V, xt)
        test_equal_logits_go_to_the_lower_id(V, xt)
        for offset in (1, 7):
            _check(_logits(rng, 3, V, xt, V + 13, offset), rng.integers(0, V, (3, 2)).astype(np.int32), 4, 1.0)
        for rows in (256, 257) if (V, xt) == (16385, "f32") else ():
            _check(_logits(rng, rows, V, xt), rng.integers(0, V, (rows, 1)).astype(np.int32), 3, 1.0)
    test_masked_logits(V)
    test_rows_that_have_no_distribution(V)


@pytest.mark.parametrize("top", [1, 13, 32])
def test_many_segments_and_few_keys(top):
    """Rows of many segments whose largest all lie in one of them, or in all; most
    segments masked; equal ones."""
    import torch
    V = 262149
    rng = np.random.default_rng(top)
    x = _logits(rng, 6, V, "bf16")
    x[0] = -1.0
    x[0, 70000:70040] = torch.arange(40, device="cuda").bfloat16()
    x[1] = 0.25
    x[2, 4096:] = float("-inf")
    x[3, : V - 5] = float("-inf")
    x[4] = float("-inf")
    x[4, ::8192] = 3.0
    x[5, 1::2] = float("-inf")
    _check(x, rng.integers(0, V, (6, 2)).astype(np.int32), top, 1.0)


def test_many_rows_and_rows_behind():
    """More rows than a grid's second axis; outputs given by the caller, whose
    rows behind the call's stay."""
    import moe_decode_amd as md
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(70001, 33, generator=g, device="cuda")
    tok = torch.randint(0, 33, (70001, 1), generator=g, device="cuda", dtype=torch.int32)
    ids = torch.full((70002, 3), -7, dtype=torch.int32, device="cuda")
    ent = torch.full((70002,), -7.0, device="cuda")
    r = md.token_logprobs(x, tok, 3, top_ids=ids[:70001], entropy=ent[:70001])
    lp = torch.log_softmax(x.double(), 1)
    assert (r.logprobs - lp.gather(1, tok.long())).abs().max() < 2e-6      # 10 u |lp| (up to 9) and 50 u
    assert torch.equal(ids[:70001], torch.sort(x, dim=1, descending=True, stable=True).indices[:, :3].int())
    assert (ids[70001] == -7).all() and ent[70001] == -7.0
    assert torch.equal(md.token_logprobs(x[69999:70000], tok[69999:70000], 3).entropy, ent[69999:70000])
    none = md.token_logprobs(x[:0], tok[:0], 3)
    assert none.logprobs.shape == (0, 1) and none.top_ids.shape == (0, 3)


def test_captured_calls_follow_their_inputs():
    import moe_decode_amd as md
    import torch
    rng = np.random.default_rng(2)
    x, tok = _logits(rng, 5, 40001, "bf16"), torch.zeros(5, 2, dtype=torch.int32, device="cuda")
    md.token_logprobs(x, tok, 8)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        r = md.token_logprobs(x, tok, 8)
    for i in range(4):
        x.copy_(_logits(np.random.default_rng(10 + i), 5, 40001, "bf16"))
        tok.fill_(17 * i)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(r, md.token_logprobs(x, tok, 8)):
            assert torch.equal(a, b)
