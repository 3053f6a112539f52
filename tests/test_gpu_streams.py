"""Calls with `stream=` while other work of the current stream takes memory: a
call's workspace and outputs stay its own until its kernels are done."""
import numpy as np
import pytest

from .gpu_common import dense_matrix, moe_layer, require_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _calls():
    """name -> (call of input i and a stream, its workspace's bytes)"""
    import moe_decode_amd as md
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    rng = np.random.default_rng(5)

    def randn(*shape):
        return [torch.randn(*shape, generator=g, device="cuda") for _ in range(2)]
    T, N, K = 100, 320, 1024
    W = md.DevQMatrix("i8_row", N, K, torch.from_numpy(rng.integers(-127, 128, N * K).astype(np.int8)).cuda(),
                      torch.from_numpy(rng.uniform(1e-3, 1e-2, N).astype(np.float32)).cuda())
    x = randn(T, K)
    L, Hkv, dim, page = 20000, 2, 128, 64
    n = -(-L // page)
    c = md.KVCache(torch.randint(-127, 128, (n, Hkv, page, dim), generator=g, dtype=torch.int8, device="cuda"),
                   torch.randint(-127, 128, (n, Hkv, dim, page), generator=g, dtype=torch.int8, device="cuda"),
                   torch.full((n, Hkv), 0.01, device="cuda"), torch.full((n, Hkv), 0.01, device="cuda"))
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    b = md.KVBatch(i32([0, 1]), i32([L]), i32([list(range(n))]), 1, L)
    q = randn(1, 8, dim)
    layer, gate = moe_layer("c0"), dense_matrix("c1", "q")
    xl, xg = randn(3, layer.H), randn(2, gate.cols)
    return {
        "i8_linear": (lambda i, st: md.i8_linear(W, x[i], stream=st), md.i8_linear_workspace_size(W, T)),
        "kv_attention": (lambda i, st: md.kv_attention(c, b, q[i], stream=st),
                         md.kv_attention_workspace_size(c, b, 1, 8)),
        "moe_layer_forward": (lambda i, st: md.moe_layer_forward(layer, xl[i], stream=st), md.moe_workspace_size(layer, 3)),
        "qgemv": (lambda i, st: md.qgemv(gate, xg[i], stream=st), md.qgemv_workspace_size(gate, 2)),
    }


@pytest.mark.parametrize("name", ["i8_linear", "kv_attention", "moe_layer_forward", "qgemv"])
def test_workspace_and_output_on_a_given_stream(name):
    import torch
    call, nbytes = _calls()[name]
    say(f"[streams] {name}, workspace {nbytes}")
    want = [call(i, None) for i in range(2)]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    now = torch.cuda.current_stream()
    for turn in range(3):
        got = []
        for i, st in enumerate(sides):
            st.wait_stream(now)
            with torch.cuda.stream(st):
                torch.cuda._sleep(20_000_000)       # the kernels start well after the call has returned
            got.append(call(i, st))
            # tensors of the current stream, of the sizes that the call took and let go
            taken = [torch.full((max(nbytes, 1),), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
            taken += [torch.full_like(got[-1], 9.0) for _ in range(3)]
        for st in sides:
            now.wait_stream(st)
        for i in range(2):
            assert torch.equal(got[i], want[i]), (turn, i)
        assert all(bool((t == 255).all()) for t in taken[:3]) and all(bool((t == 9.0).all()) for t in taken[3:])
        # an output let go while the current stream still reads it is not given to the next call's
        torch.cuda._sleep(20_000_000)
        copy = [t.clone() for t in got]
        del got
        again = [call(i, st) for i, st in enumerate(reversed(sides))]
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(copy[i], want[i]) and torch.equal(again[i], want[i]), (turn, i)
