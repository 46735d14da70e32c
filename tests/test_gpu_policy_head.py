"""The policy head example end to end: quantizers, block-wise GEMMs, log probabilities and
their gradient, against the same step in FP32 autograd on the unquantized operands."""
import pytest
import torch

from tests.oracle_helpers import gpu_ready

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,hidden,vocab", [(37, 256, 1040), (509, 1024, 4096)])
def test_step(tokens, hidden, vocab):
    m = gpu_ready()
    from examples.policy_head import policy_step, sample
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x = torch.randn(tokens, hidden, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(vocab, hidden, generator=g, device="cuda") * 0.05).to(torch.bfloat16)
    picked, old = sample(x, w, 0.9, g)
    adv = torch.randn(tokens, generator=g, device="cuda")
    r = policy_step(x, w, picked, old, adv, 0.9)
    assert m.device_status() == m.OK
    xf, wf = x.float().requires_grad_(), w.float().requires_grad_()
    logp = torch.log_softmax(xf @ wf.t() / 0.9, dim=1)
    lp = logp.gather(1, picked[:, None])[:, 0]
    ent = -(logp.exp() * logp).sum(1)
    # the sampler's and the learner's grids differ from BF16, and from each other, by E4M3's
    # 2^-4 a value at most: over a logit's sum of squares a few per cent of its size (about 1.5)
    assert 0 < r["drift"].item() < 0.15
    assert (r["logprob"] - lp).abs().mean().item() < 0.15
    assert (r["entropy"] - ent).abs().mean().item() < 0.1
    (-(adv * (lp - old).exp()) - 0.01 * ent).mean().backward()
    for got, want in ((r["grad_hidden"].float(), xf.grad), (r["grad_weight"], wf.grad)):
        cos = torch.nn.functional.cosine_similarity(got.flatten(), want.flatten(), dim=0).item()
        assert cos > 0.97, cos      # 1 - a few times (2^-4)^2 / 3, and the changed ratios
