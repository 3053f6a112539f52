"""Norms and rotation of queries and keys on the GPU, within the bound derived in
step_model.py of the definition in 64 bits."""
import numpy as np
import pytest

from . import step_model as M
from .gpu_common import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _make(rng, rows, heads, D, xt):
    """Rows of a wider tensor, as a projection leaves them."""
    import torch
    x = torch.from_numpy(rng.standard_normal((rows, heads + 3, D)).astype(np.float32)).cuda().to(_dt(xt))
    return x[:, 1:heads + 1] if D % 8 == 0 else x


def _check(rng, rows, hq, hk, D, rot, inter, norm, xt, yt, pos, factor=1.0, eps=1e-6, inplace=False):
    import moe_decode_amd as md
    import torch
    q, k = _make(rng, rows, hq, D, xt), _make(rng, rows, max(hk, 1), D, xt)
    q[rows // 2] *= 100.0
    k[0] *= 1e-3
    inv = (10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32)
    qw, kw = [(1 + 0.3 * rng.standard_normal(D)).astype(np.float32) if norm else None for _ in range(2)]
    if norm == "q":
        kw = None
    want_q = M.rope(q.float().cpu().numpy(), qw, eps, pos, inv, inter, factor, yt)
    want_k = M.rope(k.float().cpu().numpy(), kw, eps, pos, inv, inter, factor, yt)
    dev = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    kw_ = dict(q_weight=dev(qw), k_weight=dev(kw), eps=eps, interleaved=inter, factor=factor)
    if inplace:
        wide_q, wide_k = q._base.clone(), k._base.clone()
        yq, yk = md.qk_norm_rope(q, k if hk else None, dev(pos), dev(inv), q_out=q, k_out=k if hk else None, **kw_)
        assert yq is q
        for was, now, n in ((wide_q, q._base, hq), (wide_k, k._base, hk)):     # what lies around the heads stays
            assert torch.equal(was[:, 0], now[:, 0]) and torch.equal(was[:, n + 1:], now[:, n + 1:])
    else:
        yq, yk = md.qk_norm_rope(q, k if hk else None, dev(pos), dev(inv), out_dtype=_dt(yt), **kw_)
    for got, (y, tol) in [(yq, want_q)] + ([(yk, want_k)] if hk else []):
        assert got.dtype == _dt(yt)
        err = np.abs(got.float().cpu().numpy() - y)
        assert (err <= tol).all(), (np.argwhere(err > tol)[:4].tolist(), float((err / tol).max()))
    if not hk:
        assert yk is None


@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (256, 256), (8, 8), (80, 80), (96, 48), (192, 192), (256, 64),
                                   (128, 0), (64, 16), (248, 240)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rows,hq,hk", [(1, 4, 1), (37, 7, 3)])
def test_widths_and_layouts(D, rot, inter, rows, hq, hk):
    rng = np.random.default_rng(D + rot + rows)
    pos = rng.integers(0, 5000, rows).astype(np.int32)
    for norm, xt, yt in [(True, "f32", "f32"), (None, "bf16", "bf16"), ("q", "bf16", "f32"), (True, "f32", "bf16")]:
        _check(rng, rows, hq, hk, D, rot, inter, norm, xt, yt, pos)


@pytest.mark.parametrize("rows,hq,hk", [(1, 1, 0), (1, 64, 8), (2, 1024, 256), (3000, 2, 1), (1025, 16, 2)])
def test_grids(rows, hq, hk):
    rng = np.random.default_rng(rows)
    _check(rng, rows, hq, hk, 64, 64, False, True, "bf16", "bf16", np.arange(rows, dtype=np.int32))


def test_far_positions_negative_ones_factor_and_eps():
    rng = np.random.default_rng(5)
    pos = np.array([2 ** 31 - 1, -2 ** 31, -1, 0, 1 << 20, 999999937, -77777777], np.int32)
    _check(rng, 7, 3, 2, 128, 128, False, True, "f32", "f32", pos, factor=1.37, eps=0.1)
    _check(rng, 7, 3, 2, 128, 64, True, None, "f32", "f32", pos, factor=-0.5)


@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
def test_in_place(xt, inter):
    rng = np.random.default_rng(6)
    _check(rng, 65, 6, 2, 128, 96, inter, True, xt, xt, np.arange(65, dtype=np.int32), inplace=True)


def test_nothing_to_do_and_the_same_bits_again():
    import moe_decode_amd as md
    import torch
    inv = torch.ones(32, device="cuda")
    a, b = md.qk_norm_rope(torch.empty(0, 4, 64, device="cuda"), torch.empty(0, 2, 64, device="cuda"),
                           torch.empty(0, dtype=torch.int32, device="cuda"), inv)
    assert a.shape == (0, 4, 64) and b.shape == (0, 2, 64)
    q, k = torch.randn(33, 4, 64, device="cuda"), torch.randn(33, 2, 64, device="cuda")
    pos = torch.arange(33, dtype=torch.int32, device="cuda")
    w = torch.rand(64, device="cuda")
    first = md.qk_norm_rope(q, k, pos, inv, w, w)
    one = md.qk_norm_rope(q[20:21], k[20:21], pos[20:21], inv, w, w)     # a row does not depend on the others
    assert torch.equal(first[0][20:21], one[0]) and torch.equal(first[1][20:21], one[1])


def test_a_nan_stays_in_its_row_and_head():
    import moe_decode_amd as md
    import torch
    q, k = torch.randn(9, 4, 128, device="cuda"), torch.randn(9, 2, 128, device="cuda")
    pos, inv = torch.arange(9, dtype=torch.int32, device="cuda"), torch.rand(64, device="cuda")
    w = torch.rand(128, device="cuda")
    clean = md.qk_norm_rope(q, k, pos, inv, w, w)
    q[4, 1, 7], k[2, 0, 127], q[0, 3, 0] = float("nan"), float("inf"), float("-inf")
    got = md.qk_norm_rope(q, k, pos, inv, w, w)
    bad = [torch.zeros(9, 4, dtype=torch.bool, device="cuda"), torch.zeros(9, 2, dtype=torch.bool, device="cuda")]
    bad[0][4, 1] = bad[0][0, 3] = bad[1][2, 0] = True
    for c, g, b in zip(clean, got, bad):
        assert torch.equal(c[~b], g[~b]) and g[b].isnan().any(-1).all()
