"""Results in place of the operands they are made from, at widths whose rows share 32-byte sectors
and take the narrow accesses, with launches before and behind on the same memory. The same calls
with buffers of their own and a wait after each give the bits."""
import os
import subprocess
import sys

import pytest
import torch

from tests.oracle_helpers import gpu_ready

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def m():
    mod = gpu_ready()
    yield mod
    assert mod.device_status() == mod.OK


# a warp a token and the CTA, of accesses of 2 to 16 bytes, of few and many rows a token
@pytest.mark.parametrize("tokens,k,dtype,cols", [
    (1999, 4, BF16, 97), (1999, 3, BF16, 1033), (700, 8, BF16, 2050), (700, 5, BF16, 2052),
    (1203, 2, BF16, 200), (300, 1, BF16, 8200), (1203, 4, BF16, 136), (500, 8, BF16, 2056),
    (1999, 4, FP32, 97), (1203, 3, FP32, 1033), (700, 6, FP32, 258), (500, 2, FP32, 2052)])
def test_rows_gradient_in_place(m, tokens, k, dtype, cols):
    g = torch.Generator().manual_seed(cols)
    ids = torch.randint(-1, 12, (3, tokens, k), generator=g).to(DEV)
    x0 = torch.randn(tokens, cols, generator=g).to(dtype).to(DEV)
    w = torch.rand(tokens, k, generator=g).to(DEV)

    def chain(in_place):
        def wait():
            if not in_place:
                torch.cuda.synchronize()

        x, kept = x0.clone(), []
        for i in range(9):
            plan = m.route(ids[i % 3], 12)
            y = m.dispatch(x, plan, w)
            wait()
            y, grad_w = m.combine_backward(x, y, plan, w, out=y if in_place else None)
            wait()
            y, again = m.combine_backward(x, y, plan, grad_w, out=y if in_place else None)
            wait()
            kept += [grad_w, again]
            x = m.combine(y, plan, w, out=x if in_place else None)
            wait()
            x /= x.float().abs().amax()   # stays in range
        return kept + [x, y]

    for a, b in zip(chain(True), chain(False)):
        assert torch.isfinite(a).all() and torch.equal(a, b)


@pytest.mark.parametrize("rows,width,start", [(333, 96, 0), (333, 96, 8), (64, 4128, 0),
                                              (64, 4128, 8), (2000, 32, 8)])
def test_activation_in_place_of_its_rows_gradient(m, rows, width, start):
    """Buffers that start on 32 bytes, and on 16 alone."""
    g = torch.Generator().manual_seed(width)
    kept = [m.swiglu(torch.randn(rows, 2 * width, generator=g).to(BF16).to(DEV))
            for _ in range(2)]
    dh0 = torch.randn(rows, width, generator=g).to(BF16).to(DEV)

    def buffer():
        return torch.empty(start + rows * width, dtype=BF16, device=DEV)[start:].view(rows, width)

    def chain(in_place):
        dh, grads = buffer().copy_(dh0), []
        for i in range(10):
            grad, h = m.swiglu_backward(dh, *kept[i % 2][1:], recompute=True,
                                        out_h=dh if in_place else buffer())
            grads.append(grad)
            dh = h     # the next call's gradient
            if not in_place:
                torch.cuda.synchronize()
        return grads + [dh]

    for a, b in zip(chain(True), chain(False)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("start", [0, 8])
def test_activation_in_place_of_rows_gradient_past_range(m, start):
    """Threads that make their results again, beside those that do not: infinities, NaN and products
    past FP32 among the values."""
    rows, width = 257, 96
    g = torch.Generator().manual_seed(5)
    x = torch.randn(rows, 2 * width, generator=g)
    x[::7, 3], x[::11, 40], x[::13, width + 70] = 3.39e38, -3.39e38, 3.39e38
    x[5, 1], x[6, width + 1], x[8, 2] = float("nan"), float("inf"), -80
    dh0 = torch.randn(rows, width, generator=g)
    dh0[::5, ::9], dh0[9, 9], dh0[10, 10] = 2.0 ** 100, float("nan"), -float("inf")
    dh0 = dh0.to(BF16).to(DEV)
    kept = m.swiglu(x.to(BF16).to(DEV))[1:]
    want, want_h = m.swiglu_backward(dh0, *kept, recompute=True)
    assert not torch.isfinite(want).all() and not torch.isfinite(want_h).all()
    dh = torch.empty(start + rows * width, dtype=BF16, device=DEV)[start:].view(rows, width)
    dh.copy_(dh0)
    got, h = m.swiglu_backward(dh, *kept, recompute=True, out_h=dh)
    bits = lambda t: t.view(torch.int16)  # noqa: E731
    assert h is dh and torch.equal(bits(got), bits(want)) and torch.equal(bits(h), bits(want_h))
    alone, none = m.swiglu_backward(dh0, *kept)
    assert none is None and torch.equal(bits(alone), bits(want))


def test_without_programmatic_launches():
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", __file__, "-k", "rows_gradient"],
                       env=dict(os.environ, MXFP8_PDL="0"), capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stdout[-2000:]
