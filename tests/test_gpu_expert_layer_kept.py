"""What the expert layer example keeps between its passes: with no intermediates, what the backward
pass reads and nothing else, with the same results."""
import os
import sys

import pytest
import torch

from tests.oracle_helpers import gpu_ready

pytestmark = pytest.mark.gpu
DEV, ROOT = "cuda", os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
T, H, F, E, K = 203, 256, 160, 6, 2


class Watched(dict):
    def __init__(self, *a):
        super().__init__(*a)
        self.read = set()

    def __getitem__(self, key):
        self.read.add(key)
        return super().__getitem__(key)


def test_kept_is_what_the_backward_pass_reads():
    m = gpu_ready()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import expert_layer as X
    g = torch.Generator().manual_seed(2)
    bf16 = lambda *s: (torch.randn(*s, generator=g) * 0.1).to(torch.bfloat16).to(DEV)  # noqa: E731
    x, grad_out, router = bf16(T, H), bf16(T, H), bf16(E, H).float()
    experts = X.quantize_experts(bf16(E, 2 * F, H), bf16(E, H, F))
    out, kept = X.forward(x, router, experts, K, intermediates=False)
    watched = Watched(kept)
    grads = X.backward(grad_out, x, router, experts, watched)
    assert watched.read == set(kept)
    # the activation's input in MXFP8 alone: no BF16 tensor of the segments' rows but the result y
    rows = kept["y"].shape[0]
    assert [k for k, v in kept.items() if torch.is_tensor(v) and v.shape[0] == rows
            and v.dtype == torch.bfloat16] == ["y"]
    assert kept["codes"].shape == (rows, 2 * F) and kept["codes"].dtype == torch.uint8
    same, more = X.forward(x, router, experts, K)
    assert torch.equal(out, same) and set(more) == set(kept) | {"gate_up", "h"}
    again = X.backward(grad_out, x, router, experts, more)
    for k in grads:
        assert torch.equal(grads[k], again[k]), k
    assert m.device_status() == m.OK
