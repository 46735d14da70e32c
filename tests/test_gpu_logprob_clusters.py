"""Token log probabilities of few long rows, whose parts several CTAs of a cluster share:
2, 4 and 8 parts, with few and many alternatives, against the float64 oracle."""
import pytest
import torch

from tests.oracle_helpers import gpu_ready
from tests.test_gpu_logprob import check_forward, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    mod = gpu_ready()
    yield mod
    assert mod.device_status() == mod.OK


@pytest.mark.parametrize("rows,vocab", [(1, 4099), (7, 8200), (2, 16391), (40, 9001), (3, 65537)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("top", [0, 1, 17, 32])
def test_parts_of_a_row(m, rows, vocab, dtype, top):
    x, t = make(rows * 7 + vocab + top, rows, vocab, dtype, vocab + 5, 3)
    check_forward(m, x, t, 0.8, top)
    x[0, : vocab // 2] = -float("inf")      # the first parts hold nothing
    x[-1, vocab // 2:] = 1.5                # ties across the last parts
    check_forward(m, x, t, 0.8, top)
