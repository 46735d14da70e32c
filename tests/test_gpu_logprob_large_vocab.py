"""Sums over very large vocabularies. A thread adds up n = max(256, vocab / 256) terms at most in
order, each rounding by 2^-24 of the running sum, then some 64 steps join the threads and the
CTAs; a term itself is off by 2^-22 (its power of two) and by its exponent's rounding, 2^-20 in
all: |error of log S| <= (n + 64) 2^-24 + 2^-20. One value far above the others is the hardest
for a running sum: what is added to it falls below its last bit."""
import pytest
import torch

from tests.oracle_helpers import gpu_ready

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def m():
    mod = gpu_ready()
    yield mod
    assert mod.device_status() == mod.OK


@pytest.mark.parametrize("rows,vocab", [(1, (1 << 26) + 5), (2, 1 << 24), (170, (1 << 21) + 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("peak", [0.0, 16.0])
def test_log_sum(m, rows, vocab, dtype, peak):
    g = torch.Generator(device=DEV).manual_seed(vocab)
    x = torch.randn(rows, vocab, generator=g, device=DEV).to(dtype)
    if peak:
        x[:, 0] = peak
    t = torch.zeros(rows, dtype=torch.int64, device=DEV)
    r = m.token_logprobs(x, t)
    tol = (max(256, -(-vocab // 256)) + 64) * 2.0 ** -24 + 2.0 ** -20
    for i in range(0, rows, 17):
        z = x[i].double()
        top = z.max()
        log_sum = torch.logsumexp(z - top, 0)
        assert r.stats[i, 0].double() == top
        assert (r.stats[i, 1].double() - log_sum).abs() <= tol
        want = z[0] - top - log_sum
        assert (r.logprob[i].double() - want).abs() <= tol + want.abs() * 2.0 ** -22
