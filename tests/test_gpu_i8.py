"""The 8-bit products on the GPU: codes and scales equal to the definition's,
outputs within the roundings of their last steps, whatever the number of
tokens (each launch shape's borders), on rows with special values."""
import numpy as np
import pytest

from .gpu_common import require_gpu, say
from .kv_model import HALF, codes_of, step_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def _dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _rows(T, K, seed):
    """Rows of very different sizes, channels far above the others."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, K)) * np.exp(rng.uniform(-6, 6, (T, 1)))
    x[:, :: max(1, K // 5)] *= 20
    return x.astype(np.float32)


def _codes(x):
    s = np.array([step_of(a) for a in np.abs(x).max(1)], np.float32)
    return codes_of(x, s[:, None]), s


@pytest.mark.parametrize("T,K", [(1, 256), (3, 256), (5, 512), (2, 768), (7, 2048), (3, 2304), (4, 6144), (2, 6400),
                                 (5, 16384), (1, 16384)])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_codes_are_the_definitions(T, K, xt):
    import moe_decode_amd as md
    x = _dev(_rows(T, K, 10 * T + K), _dt(xt))
    codes, scales = md.i8_quantize(x)
    want, s = _codes(x.float().cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), want)


def test_codes_next_to_the_borders():
    """Every k + 1/2 times a scale, and its fp32 neighbours; scales over the
    whole range, subnormal steps among them."""
    import moe_decode_amd as md
    rows = []
    for top in (127.0, 1.0, 3.3e38, 1e-30, 2.0 ** -110, 1e-37, 1.2e-38, 3e-41, 190 * 2.0 ** -149, 100 * 2.0 ** -149,
                63 * 2.0 ** -149, 2.0 ** -149):
        top = np.float32(top)
        s = step_of(top)
        b = (np.arange(-126.5, 127.0, 3.0) * np.float64(s)).astype(np.float32)
        b = b[np.abs(b) <= top]
        row = np.concatenate([b, np.nextafter(b, np.float32(np.inf)), np.nextafter(b, np.float32(-np.inf))])
        row = row[np.abs(row) <= top][:255]
        rows.append(np.concatenate([[top], row, np.zeros(255 - len(row), np.float32)]).astype(np.float32))
    x = np.stack(rows)
    codes, scales = md.i8_quantize(_dev(x))
    want, s = _codes(x)
    assert np.array_equal(scales.cpu().numpy(), s)
    for i in range(len(rows)):
        assert np.array_equal(codes.cpu().numpy()[i], want[i]), (i, float(x[i, 0]))


def _product(x, w, ws, b, out):
    """The result and its bound: int32 to fp32, two scale products, the bias add
    (u = 2^-24 each, relative), and the output's own rounding.  The factors of
    the products after a rounding: under 1 + 4 u, covered by the 1.01."""
    q, s = _codes(x)
    acc = q.astype(np.int64) @ w.astype(np.int64).T
    p = acc * s.astype(np.float64)[:, None] * ws.astype(np.float64)
    y = p if b is None else p + b.astype(np.float64)
    return y, 1.01 * (3 * 2.0 ** -24 * np.abs(p) + 2.0 ** -24 * np.abs(y)) + HALF[out] * np.abs(y) + 1e-44


# the last token counts of a launch shape and the first of the next, and widths around a tile's
SHAPES = [(1, 1, 256), (1, 256, 2048), (2, 17, 512), (3, 40, 16384), (4, 20, 16384), (4, 100, 6144), (5, 50, 16384), (15, 33, 1024), (16, 64, 1280), (17, 31, 256), (32, 100, 4352),
          (33, 48, 768), (64, 130, 2048), (65, 64, 512), (100, 200, 768), (127, 65, 256), (128, 1500, 256),
          (2, 15, 256), (7, 33, 768), (8, 70, 2048), (9, 40, 2048), (8, 90, 2304), (8, 8192, 2048), (8, 8193, 2048),
          (129, 129, 1024), (300, 1000, 512), (70, 64, 4096), (500, 100, 2048), (1000, 1111, 256), (2100, 2049, 256)]


@pytest.mark.parametrize("T,N,K", SHAPES)
@pytest.mark.parametrize("xt,out,bias", [("f32", "f32", True), ("bf16", "bf16", False), ("f32", "bf16", True),
                                         ("bf16", "f32", False)])
def test_linear(T, N, K, xt, out, bias):
    import moe_decode_amd as md
    import torch
    say(f"[i8] T={T} N={N} K={K} {xt} -> {out}")
    rng = np.random.default_rng(T * 7 + N)
    w = rng.integers(-128, 128, (N, K)).astype(np.int8)
    ws = rng.uniform(1e-3, 1e-2, N).astype(np.float32)
    b = rng.standard_normal(N).astype(np.float32) if bias else None
    x = _dev(_rows(T, K, T + K), _dt(xt))
    W = md.DevQMatrix("i8_row", N, K, _dev(w).view(-1), _dev(ws))
    guard = torch.full((T + 1, N), 7.0, dtype=_dt(out), device="cuda")
    y = md.i8_linear(W, x, bias=None if b is None else _dev(b), y=guard[:T])
    ref, tol = _product(x.float().cpu().numpy(), w, ws, b, out)
    got = y.double().cpu().numpy()
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist())
    assert bool((guard[T] == 7.0).all())
    # the two halves are the whole, and a token's result does not depend on the others
    codes, scales = md.i8_quantize(x)
    assert torch.equal(md.i8_matmul(W, codes, scales, bias=None if b is None else _dev(b), out_dtype=_dt(out)), y)
    t = T // 2
    one = md.i8_linear(W, x[t:t + 1].contiguous(), bias=None if b is None else _dev(b), out_dtype=_dt(out))
    assert torch.equal(one[0], y[t])


@pytest.mark.parametrize("T", [6, 70])
def test_rows_that_are_not_finite_and_rows_of_zeros(T):
    import moe_decode_amd as md
    import torch
    N, K = 40, 512
    x = _rows(T, K, 5)
    x[1], x[2, 3], x[4, 500], x[5, 0] = 0, np.inf, np.nan, -np.inf
    w = np.random.default_rng(1).integers(-127, 128, (N, K)).astype(np.int8)
    w[7] = 0
    ws, b = np.full(N, 0.01, np.float32), np.arange(N, dtype=np.float32)
    W = md.DevQMatrix("i8_row", N, K, _dev(w).view(-1), _dev(ws))
    codes, scales = md.i8_quantize(_dev(x))
    for r in (2, 4, 5):
        assert bool(torch.isnan(scales[r])) and not bool(codes[r].any())
    assert float(scales[1]) == 0.0 and not bool(codes[1].any())
    y = md.i8_linear(W, _dev(x), bias=_dev(b)).cpu().numpy()
    assert np.isnan(y[[2, 4, 5]]).all()
    assert np.array_equal(y[1], b)
    rest = [r for r in range(T) if r not in (2, 4, 5)]
    ref, tol = _product(x[rest], w, ws, b, "f32")
    assert (np.abs(y[rest] - ref) <= tol).all()


def test_no_tokens_and_refused_tensors():
    import moe_decode_amd as md
    import torch
    W = md.DevQMatrix("i8_row", 8, 256, torch.zeros(8 * 256, dtype=torch.int8, device="cuda"),
                      torch.ones(8, device="cuda"))
    assert md.i8_linear(W, torch.zeros(0, 256, device="cuda")).shape == (0, 8)
    x = torch.zeros(4, 256, device="cuda")
    for bad in (x.half(), x.double()):
        with pytest.raises((TypeError, ValueError)):
            md.i8_linear(W, bad)
    with pytest.raises(ValueError):
        md.i8_linear(W, torch.zeros(4, 512, device="cuda")[:, ::2])
    with pytest.raises(ValueError):
        md.i8_linear(W, torch.zeros(4, 512, device="cuda"))
    with pytest.raises(ValueError):
        md.i8_linear(W, x, bias=torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError):
        md.i8_linear(W, x, y=torch.zeros(4, 9, device="cuda"))
    with pytest.raises(ValueError):
        md.i8_linear(W, x.cpu())
    with pytest.raises(md.MDError) as e:
        md.i8_linear(W, torch.zeros(9, 256, device="cuda"), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.name == "MD_ERR_WORKSPACE"


def test_on_a_stream_and_in_a_graph():
    """A call on a side stream, and a captured one replayed with other inputs."""
    import moe_decode_amd as md
    import torch
    T, N, K = 37, 72, 768
    rng = np.random.default_rng(9)
    W = md.DevQMatrix("i8_row", N, K, _dev(rng.integers(-127, 128, (N, K)).astype(np.int8)).view(-1),
                      _dev(rng.uniform(1e-3, 1e-2, N).astype(np.float32)))
    xs = [_dev(_rows(T, K, i)) for i in range(4)]
    want = [md.i8_linear(W, x) for x in xs]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = md.i8_linear(W, xs[0])
    st.synchronize()
    assert torch.equal(got, want[0])
    x, y = xs[0].clone(), torch.empty(T, N, device="cuda")
    ws = torch.empty(md.i8_linear_workspace_size(W, T), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        md.i8_linear(W, x, y=y, workspace=ws)
    for i in (1, 2, 3, 1):
        x.copy_(xs[i])
        g.replay()
        assert torch.equal(y, want[i])
        assert torch.equal(md.i8_linear(W, xs[i]), want[i])
        torch.cuda.synchronize()
