"""A mixture-of-experts layer in MXFP8, forward and backward, from the router's choice to the
gradients of the tokens, the router and the experts' weights.

The routed tokens of "End-to-End MXFP8 RL on Blackwell" (section "A held-out workload, and end to
end", Table 4: a model with 128 experts, 8 a token) go through it like this:

    route -> dispatch into MXFP8 -> gate_up product -> gated activation, its input kept in 8 bits
          -> down product -> combine

The router stays in higher precision, as on the pages. What the backward pass needs is kept in 8
bits where the GEMMs read it so: the routed tokens' column copy, the activation's input; the down
product's result is kept for the gradient of the router's weights.

    python examples/expert_layer.py --tokens 1021 --hidden 2048 --width 768 --experts 128 --top 8
"""
import argparse
import os
import sys
from typing import NamedTuple

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp8_block_scaled_05_gb300 as m  # noqa: E402


class Experts(NamedTuple):
    """Quantized weights, row-wise for the forward products, column-wise for the gradients'."""
    gate_up: tuple     # of [experts, 2 * width, hidden]: codes and scales
    gate_up_t: tuple
    down: tuple        # of [experts, hidden, width]
    down_t: tuple


def quantize_experts(gate_up, down):
    return Experts(m.quantize_batched(gate_up, m.ROW), m.quantize_batched(gate_up, m.COL),
                   m.quantize_batched(down, m.ROW), m.quantize_batched(down, m.COL))


def forward(x, router, experts, top, intermediates=True):
    """x: BF16 [tokens, hidden], router: float32 [experts, hidden]. Returns the result (BF16
    [tokens, hidden]) and what the backward pass reads; with intermediates, for a look at each step,
    also the activation's input and result in BF16, which it does not read."""
    logits = x.float() @ router.t()
    none = torch.full((x.shape[0],), -1, device=x.device)
    chosen = m.token_logprobs(logits, none, top=top)
    weights = chosen.top_logprob.exp()
    plan = m.route(chosen.top_id, router.shape[0])
    xr, xrs, xc, xcs = m.quantize_dispatch_dual(x, plan)
    gate_up = m.grouped_gemm(xr, xrs, *experts.gate_up, plan.offsets, m.FPROP)
    act = m.swiglu(gate_up)
    y = m.grouped_gemm(*m.quantize_grouped(act.h, plan.offsets, m.ROW), *experts.down,
                       plan.offsets, m.FPROP)
    out = m.combine(y, plan, weights)
    kept = dict(logits=logits, chosen=chosen, weights=weights, plan=plan, x_col=(xc, xcs),
                codes=act.codes, scales=act.scales, y=y)
    if intermediates:
        kept.update(gate_up=gate_up, h=act.h)
    return out, kept


def backward(grad_out, x, router, experts, kept):
    """Gradients of x (BF16), router, gate_up and down (float32)."""
    plan, weights, chosen = kept["plan"], kept["weights"], kept["chosen"]
    off = plan.offsets
    dyr, dyrs, dyc, dycs = m.quantize_dispatch_dual(grad_out, plan, weights)
    _, grad_weights = m.combine_backward(grad_out, kept["y"], plan, weights, grad_rows=False)
    grad_h = m.grouped_gemm(dyr, dyrs, *experts.down_t, off, m.DGRAD)
    grad_gate_up, h = m.swiglu_backward(grad_h, kept["codes"], kept["scales"], recompute=True)
    grad_down = m.grouped_gemm(dyc, dycs, *m.quantize_grouped(h, off, m.COL), off, m.WGRAD,
                               m.OUT_FP32)
    dgr, dgrs, dgc, dgcs = m.quantize_grouped_dual(grad_gate_up, off)
    grad_rows = m.grouped_gemm(dgr, dgrs, *experts.gate_up_t, off, m.DGRAD)
    grad_x = m.combine(grad_rows, plan)
    grad_gate = m.grouped_gemm(dgc, dgcs, *kept["x_col"], off, m.WGRAD, m.OUT_FP32)
    # the weights are exponentials of the chosen experts' log probabilities
    tokens = x.shape[0]
    none = torch.full((tokens,), -1, device=x.device)
    grad_logits = m.token_logprobs_backward(
        kept["logits"], none, chosen.stats, chosen.entropy,
        torch.zeros(tokens, device=x.device), top_id=chosen.top_id,
        grad_top=grad_weights * weights)
    grad_x = (grad_x.float() + grad_logits @ router).to(torch.bfloat16)
    return dict(x=grad_x, router=grad_logits.t() @ x.float(), gate_up=grad_gate, down=grad_down,
                weights=grad_weights, h=grad_h, gate_up_rows=grad_gate_up, rows=grad_rows,
                h_again=h, logits=grad_logits)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=1021)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--width", type=int, default=768)
    ap.add_argument("--experts", type=int, default=128)
    ap.add_argument("--top", type=int, default=8)
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = rand(a.tokens, a.hidden).to(torch.bfloat16)
    router = rand(a.experts, a.hidden) * 0.02
    experts = quantize_experts((rand(a.experts, 2 * a.width, a.hidden) * 0.02).to(torch.bfloat16),
                               (rand(a.experts, a.hidden, a.width) * 0.02).to(torch.bfloat16))
    out, kept = forward(x, router, experts, a.top, intermediates=False)
    grads = backward(rand(a.tokens, a.hidden).to(torch.bfloat16), x, router, experts, kept)
    status = m.device_status()
    if status != m.OK:
        raise m.MXFP8Error(status, "expert layer")
    rows, width = kept["codes"].shape[0], kept["codes"].shape[1] // 2
    print(f"tokens {a.tokens}, hidden {a.hidden}, {a.top} of {a.experts} experts of {a.width}; "
          f"{rows} segment rows")
    print(f"kept for the activation's gradient: {(kept['codes'].numel() + kept['scales'].numel()) / 2**20:.1f} MiB "
          f"(BF16: {4 * rows * width / 2**20:.1f} MiB)")
    print("|out| %.4g, " % out.float().norm().item()
          + ", ".join(f"|grad {k}| {grads[k].float().norm().item():.4g}"
                      for k in ("x", "router", "gate_up", "down")))


if __name__ == "__main__":
    main()
