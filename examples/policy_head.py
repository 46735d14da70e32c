"""One policy-gradient step through a policy's output head in block-wise FP8.

A sampler and a learner hold the same BF16 head but quantize it with different block scales:
the sampler with FP32 scales, the learner with powers of two, as the block-wise recipe has to
on Blackwell ("End-to-End MXFP8 RL on Blackwell", section "A different grid, and drift").
The sampler proposes tokens; the learner scores the same tokens, and the difference of the
two log probabilities is the drift. The step then runs the learner's gradient: from the
policy loss to the logits, and through the head's two gradient products.

    python examples/policy_head.py --tokens 509 --hidden 2048 --vocab 16384
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp8_block_scaled_05_gb300 as m  # noqa: E402


def head(hidden, weight, scale_type):
    """logits = hidden . weight^T in block-wise FP8."""
    x, sx = m.quantize_blockwise_1d(hidden, m.ROW, scale_type)
    w, sw = m.quantize_blockwise(weight, scale_type)
    return m.blockwise_gemm(x, sx, w, sw, m.FPROP, scale_type=scale_type)


def sample(hidden, weight, temperature, generator):
    """The sampler's side: tokens drawn among each position's likeliest, and their log
    probabilities under the sampler's grid."""
    logits = head(hidden, weight, m.BW_FP32)
    none = torch.full((hidden.shape[0],), -1, device=hidden.device)
    best = m.token_logprobs(logits, none, temperature, top=m.MAX_TOP)
    pick = torch.multinomial(best.top_logprob.exp(), 1, generator=generator)
    return best.top_id.gather(1, pick)[:, 0], best.top_logprob.gather(1, pick)[:, 0]


def policy_step(hidden, weight, tokens, old_logprob, advantage, temperature=1.0,
                entropy_bonus=0.01):
    """The learner's side: forward, policy gradient and the head's gradients. Returns the drift
    (mean |log probability - the sampler's|), the entropy, and the gradients of the loss
    mean(-advantage * exp(logprob - old_logprob) - entropy_bonus * entropy) with respect to
    hidden (BF16) and weight (FP32)."""
    n = tokens.numel()
    x, sx, xt, sxt = m.quantize_blockwise_1d_dual(hidden, m.BW_POW2)
    w, sw, wt, swt = m.quantize_blockwise_dual(weight, m.BW_POW2)
    logits = m.blockwise_gemm(x, sx, w, sw, m.FPROP)
    scored = m.token_logprobs(logits, tokens, temperature)
    ratio = (scored.logprob - old_logprob).exp()
    g_logprob = -advantage * ratio / n
    g_entropy = torch.full_like(g_logprob, -entropy_bonus / n)
    # the gradient replaces the logits in place
    m.token_logprobs_backward(logits, tokens, scored.stats, scored.entropy, g_logprob, g_entropy,
                              temperature=temperature, out=logits)
    d, sd, dt, sdt = m.quantize_blockwise_1d_dual(logits, m.BW_POW2)
    grad_hidden = m.blockwise_gemm(d, sd, wt, swt, m.DGRAD)
    grad_weight = m.blockwise_gemm(dt, sdt, xt, sxt, m.WGRAD, m.OUT_FP32)
    return dict(drift=(scored.logprob - old_logprob).abs().mean(), logprob=scored.logprob,
                entropy=scored.entropy, grad_hidden=grad_hidden, grad_weight=grad_weight)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=509)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--vocab", type=int, default=16384)
    ap.add_argument("--temperature", type=float, default=1.0)
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)
    hidden = torch.randn(a.tokens, a.hidden, generator=g, device="cuda").to(torch.bfloat16)
    weight = (torch.randn(a.vocab, a.hidden, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    tokens, old = sample(hidden, weight, a.temperature, g)
    advantage = torch.randn(a.tokens, generator=g, device="cuda")
    r = policy_step(hidden, weight, tokens, old, advantage, a.temperature)
    status = m.device_status()
    if status != m.OK:
        raise m.MXFP8Error(status, "policy step")
    print(f"tokens {a.tokens}, hidden {a.hidden}, vocabulary {a.vocab}")
    print(f"drift between the two grids: mean |log probability difference| {r['drift'].item():.4f}")
    print(f"mean entropy {r['entropy'].mean().item():.3f}, |grad hidden| "
          f"{r['grad_hidden'].float().norm().item():.4g}, |grad weight| "
          f"{r['grad_weight'].norm().item():.4g}")


if __name__ == "__main__":
    main()
