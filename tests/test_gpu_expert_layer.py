"""The expert layer example: a run of the routing operators, the gated activation and the grouped
GEMMs, forward and backward. Each step is held to the oracle on the GPU's own inputs of that
step, so every tolerance is that of one operator: the GEMM gate, and the bounds that
test_gpu_routing.py and test_gpu_swiglu.py derive."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle.logprob_oracle as L
import oracle.mxfp8_oracle as O
import oracle.routing_oracle as R
import oracle.swiglu_oracle as S
from tests.oracle_helpers import assert_gemm_within, bf16_bits, gpu_ready

pytestmark = pytest.mark.gpu
DEV, ROOT = "cuda", os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
T, H, F, E, K = 203, 256, 160, 6, 2


def f64(t):
    return t.double().cpu().numpy()


def within_bf16(got, want, tol, what):
    err = np.abs(f64(got) - want)
    bound = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want) + 2.0 ** -133
    assert (err <= bound).all(), (what, np.max(err - bound))


def rows_gemm(a, w, off, what, got):
    """A grouped forward or data-gradient product of BF16 a with BF16 weights w [E, N, K]."""
    qa, sa = O.quantize(bf16_bits(a), O.ROW)
    qw, sw = zip(*(O.quantize(bf16_bits(w[e]), O.ROW) for e in range(E)))
    want, mag = np.zeros(got.shape), np.zeros(got.shape)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            want[lo:hi] = O.gemm(qa[lo:hi], sa[lo:hi], qw[e], sw[e])
            mag[lo:hi] = O.gemm_abs(qa[lo:hi], sa[lo:hi], qw[e], sw[e])
    assert_gemm_within(f64(got), want, mag, True, what)


def wgrad_gemm(dy, x, off, what, got):
    qa, sa = O.quantize(bf16_bits(dy), O.COL)
    qb, sb = O.quantize(bf16_bits(x), O.COL)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if hi == lo:
            assert not got[e].any(), what
            continue
        args = (qa[:, lo:hi], sa[:, lo // 32:hi // 32], qb[:, lo:hi], sb[:, lo // 32:hi // 32])
        assert_gemm_within(f64(got[e]), O.gemm(*args), O.gemm_abs(*args), False, what)


def test_each_step_matches_the_oracle():
    m = gpu_ready()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import expert_layer as X
    g = torch.Generator().manual_seed(0)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    router = (torch.randn(E, H, generator=g) * 0.1).to(DEV)
    w1 = (torch.randn(E, 2 * F, H, generator=g) * 0.1).to(torch.bfloat16).to(DEV)
    w2 = (torch.randn(E, H, F, generator=g) * 0.1).to(torch.bfloat16).to(DEV)
    experts = X.quantize_experts(w1, w2)
    out, kept = X.forward(x, router, experts, K)
    grad_out = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    grads = X.backward(grad_out, x, router, experts, kept)
    assert m.device_status() == m.OK

    # ---- the plan
    ids = kept["chosen"].top_id
    plan, weights = kept["plan"], kept["weights"].cpu().numpy()
    rows = R.rows_for(T, K, E)
    off, row_of, entry_of = R.route(ids.cpu().numpy(), E, rows)
    for got, want in zip(plan, (off, row_of, entry_of)):
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    logits = f64(kept["logits"])
    np.testing.assert_array_equal(ids.cpu().numpy(), np.argsort(-logits, axis=1)[:, :K])

    # ---- forward
    def spread(t, w=None):   # the dispatched rows, in BF16
        return m.dispatch(t, plan, None if w is None else kept["weights"])

    routed = spread(x)
    rows_gemm(routed, w1, off, "gate_up", kept["gate_up"])
    v = f64(kept["gate_up"])
    within_bf16(kept["h"], S.forward(v[:, :F], v[:, F:]), S.forward_error(v[:, :F], v[:, F:]), "h")
    rows_gemm(kept["h"], w2, off, "down", kept["y"])
    want, mag = R.combine(f64(kept["y"]), row_of, weights)
    within_bf16(out, want, (K + 1) * 2.0 ** -24 * mag, "out")

    # ---- backward
    dy = spread(grad_out, True)
    rows_gemm(dy, w2.transpose(1, 2).contiguous(), off, "grad_h", grads["h"])
    kept_v = O.dequantize(kept["codes"].cpu().numpy(), kept["scales"].cpu().numpy())
    a, u, d = kept_v[:, :F], kept_v[:, F:], f64(grads["h"])
    for got, want, tol in zip((grads["gate_up_rows"][:, :F], grads["gate_up_rows"][:, F:]),
                              S.backward(a, u, d), S.backward_error(a, u, d)):
        within_bf16(got, want, tol, "grad_gate_up")
    within_bf16(grads["h_again"], S.forward(a, u), S.forward_error(a, u), "h again")
    wgrad_gemm(dy, grads["h_again"], off, "grad_down", grads["down"])
    wgrad_gemm(grads["gate_up_rows"], routed, off, "grad_gate_up_w", grads["gate_up"])
    rows_gemm(grads["gate_up_rows"], w1.transpose(1, 2).contiguous(), off, "grad_rows",
              grads["rows"])
    want, mag = R.combine_weights_grad(f64(grad_out), f64(kept["y"]), row_of)
    err = np.abs(f64(grads["weights"]) - want)
    assert (err <= (H / 128 + 144) * 2.0 ** -24 * mag).all()

    # ---- the router: sums of K + 1 FP32 terms; p is off by 2^-15 of itself at most (the log sum's
    # error of 320 2^-24 + 2^-20 and the exponential's)
    g_top = (grads["weights"] * kept["weights"]).double().cpu().numpy()
    want = L.backward(logits, np.full(T, -1), 1.0, np.zeros(T), top_id=ids.cpu().numpy(),
                      g_top=g_top)
    scale = np.abs(g_top).sum(axis=1, keepdims=True)
    assert (np.abs(f64(grads["logits"]) - want) <= 2.0 ** -15 * scale).all()
    back, mag = R.combine(f64(grads["rows"]), row_of)
    via = f64(grads["logits"]) @ f64(router)
    # two BF16 roundings and an FP32 product of E terms
    via_mag = np.abs(f64(grads["logits"])) @ np.abs(f64(router))
    tol = (K + 1) * 2.0 ** -24 * mag + 2.0 ** -8 * np.abs(back) + (E + 2) * 2.0 ** -24 * via_mag
    # torch's FP32 product may run in TF32 only where that is asked for; it is not here
    within_bf16(grads["x"], back + via, tol, "grad_x")


def test_weights_gradient_by_differences():
    """The layer's result is linear in a token's combine weights, so differences of any length give
    their gradient, but for the BF16 rounding of the result (2^-8 of it, on either side)."""
    m = gpu_ready()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import expert_layer as X
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    router = (torch.randn(E, H, generator=g) * 0.1).to(DEV)
    experts = X.quantize_experts(
        (torch.randn(E, 2 * F, H, generator=g) * 0.1).to(torch.bfloat16).to(DEV),
        (torch.randn(E, H, F, generator=g) * 0.1).to(torch.bfloat16).to(DEV))
    out, kept = X.forward(x, router, experts, K)
    grad_out = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    grad_w = X.backward(grad_out, x, router, experts, kept)["weights"]
    for j in range(K):
        up = kept["weights"].clone()
        up[:, j] += 4.0
        moved = m.combine(kept["y"], kept["plan"], up)
        step = (up[:, j] - kept["weights"][:, j]).double()
        got = ((moved.double() - out.double()) * grad_out.double()).sum(dim=1) / step
        tol = ((moved.double().abs() + out.double().abs()) * grad_out.double().abs()).sum(dim=1) \
            * 1.01 * 2.0 ** -8 / step
        assert ((got - grad_w[:, j].double()).abs() <= tol).all()


def test_the_program_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "expert_layer.py"),
                        "--tokens", "131", "--hidden", "256", "--width", "96", "--experts", "12",
                        "--top", "3"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "131" in r.stdout and "grad router" in r.stdout
