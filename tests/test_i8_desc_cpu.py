"""The checks of an int8 matrix's tensors, kept while the tensors stay: another
tensor at the same address is looked at again."""
import pytest
import torch

import moe_decode_amd as md

N, K = 8, 256


def _matrix():
    return md.DevQMatrix("i8_row", N, K, torch.zeros(N * K, dtype=torch.int8), torch.ones(N))


def _shorter(W):
    W.q = W.q[:N * K // 2]


def _turned(W):
    W.q = W.q.view(N, K).t()


def _fewer_scales(W):
    W.row_scale = W.row_scale[:N - 1]


def _scales_of_another_type(W):
    W.row_scale = W.row_scale.view(torch.int32)


def _spread_scales(W):
    W.row_scale = W.row_scale[:1].expand(N)


@pytest.mark.parametrize("change", [_shorter, _turned, _fewer_scales, _scales_of_another_type, _spread_scales])
def test_a_tensor_at_the_same_address_is_checked_again(change):
    W = _matrix()
    at = W.q.data_ptr(), W.row_scale.data_ptr()
    assert md.i8_linear_workspace_size(W, 4) >= 0
    change(W)
    assert (W.q.data_ptr(), W.row_scale.data_ptr()) == at
    for _ in range(2):
        with pytest.raises(ValueError):
            md.i8_linear_workspace_size(W, 4)


def test_the_descriptor_stays_while_the_tensors_do():
    W = _matrix()
    assert md._i8_desc(W) is md._i8_desc(W)
    old = md._i8_desc(W)
    W.q = W.q.view(N, K)            # as many bytes, in the same order
    md._i8_desc(W)
    W.q = torch.zeros(N * K, dtype=torch.int8)
    assert md._i8_desc(W) is not old
    W.rows = N // 2                 # fewer rows than the tensors hold
    assert md._i8_desc(W)._obj.rows == N // 2
    W.rows = 2 * N
    with pytest.raises(ValueError):
        md._i8_desc(W)
