"""Log probabilities of many short rows on the GPU, around the size from which a row
no longer fits one step of 8 values a thread."""
import numpy as np
import pytest

from .gpu_common import require_gpu
from .test_gpu_logprob import _check, _logits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("V,stride,offset", [(1, 3, 0), (100, 101, 5), (2040, 2047, 1), (2041, 2049, 7), (2042, 2043, 7)])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_many_short_rows(V, stride, offset, xt):
    rng = np.random.default_rng(V)
    x = _logits(rng, 601, V, xt, stride, offset)
    x[5, : V // 2] = float("-inf")
    x[6] = 2.0
    _check(x, rng.integers(0, V, (601, 2)).astype(np.int32), min(V, 8), 1.3)
    _check(x, None, 0, 1.0)
