"""The token log probabilities' gradient on ids and weights at the edge of what it accepts."""
import pytest
import torch

from tests.oracle_helpers import gpu_ready
from tests.test_gpu_logprob import make

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def m():
    mod = gpu_ready()
    yield mod
    assert mod.device_status() == mod.OK


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [100, 20011])      # one CTA a row, several
def test_alternative_past_the_vocabulary(m, dtype, vocab):
    x, t = make(3, 5, vocab, dtype)
    t[:] = torch.tensor([3, 4, -1, 6, 7], device=DEV)
    r = m.token_logprobs(x, t, top=3)
    g, gt = torch.ones(5, device=DEV), torch.ones(5, 3, device=DEV)
    want = m.token_logprobs_backward(x, t, r.stats, r.entropy, g, g, r.top_id, gt)
    assert m.device_status() == m.OK
    ids = r.top_id.clone()
    ids[1, 2], ids[2, 0] = vocab, 1 << 40
    got = m.token_logprobs_backward(x, t, r.stats, r.entropy, g, g, ids, gt)
    assert m.device_status() == m.ERR_BAD_TARGET
    assert got[1].isnan().all() and got[2].isnan().all()
    for i in (0, 3, 4):
        assert torch.equal(got[i], want[i])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("weight", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("vocab", [100, 20011])
def test_empty_row_gets_zeros_whatever_its_weights(m, dtype, weight, vocab):
    x, t = make(4, 4, vocab, dtype)
    x[1], x[2] = -float("inf"), -float("inf")
    t[:] = torch.tensor([3, 4, -1, 6], device=DEV)
    r = m.token_logprobs(x, t, top=2)
    g = torch.ones(4, device=DEV)
    gt = torch.ones(4, 2, device=DEV)
    want = m.token_logprobs_backward(x, t, r.stats, r.entropy, g, g, r.top_id, gt)
    bad = g.clone()
    bad[1:3] = weight
    gt[1:3] = weight
    got = m.token_logprobs_backward(x, t, r.stats, r.entropy, bad, bad, r.top_id, gt)
    assert (got[1:3] == 0).all()
    assert torch.equal(got[0], want[0]) and torch.equal(got[3], want[3])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab,pitch", [(3, 70001, 70016), (1, 131072, 131072)])
def test_in_place_with_rows_split_over_ctas(m, dtype, rows, vocab, pitch):
    x, t = make(5, rows, vocab, dtype, pitch)
    r = m.token_logprobs(x, t, 1.0, 5)
    g = torch.randn(rows, device=DEV)
    gt = torch.randn(rows, 5, device=DEV)
    want = m.token_logprobs_backward(x, t, r.stats, r.entropy, g, g, r.top_id, gt)
    got = m.token_logprobs_backward(x, t, r.stats, r.entropy, g, g, r.top_id, gt, out=x)
    assert got.data_ptr() == x.data_ptr() and torch.equal(got, want)
