"""The gated activation at the ends of its types' ranges: kept values of 2^128, gradients whose
products pass FP32 on the way to a result that does not, and blocks near the least scale.
Tolerances as in test_gpu_swiglu.py."""
import numpy as np
import pytest
import torch

import oracle.mxfp8_oracle as O
import oracle.swiglu_oracle as S
from tests.oracle_helpers import bf16_bits, bits_to_bf16, gpu_ready, u8

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def m():
    mod = gpu_ready()
    yield mod
    assert mod.device_status() == mod.OK


def close(got, want, tol, what):
    got = got.double().cpu().numpy()
    err, tol = np.abs(got - want), tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want) + 2.0 ** -134
    assert (err <= tol).all(), (what, np.argwhere(~(err <= tol))[:4].tolist())


def check_backward(m, x, dh):
    """The gradient, and h again, of what swiglu keeps of x, against the oracle's values of the
    kept codes; results past FP32 count as infinities. Returns the kept values."""
    width = x.shape[1] // 2
    r = m.swiglu(x.to(DEV))
    codes, scales = O.quantize(bf16_bits(x), O.ROW, rule=1)
    np.testing.assert_array_equal(u8(r.codes), codes)
    np.testing.assert_array_equal(u8(r.scales), scales)
    grad, h = m.swiglu_backward(dh.to(DEV), r.codes, r.scales, recompute=True)
    kept = O.dequantize(codes, scales)
    a, u, d = kept[:, :width], kept[:, width:], dh.double().numpy()
    dg, du = S.backward(a, u, d)
    eg, eu = S.backward_error(a, u, d)
    for got, want, tol, what in ((grad[:, :width], dg, eg, "dg"), (grad[:, width:], du, eu, "du"),
                                 (h, S.forward(a, u), S.forward_error(a, u), "h")):
        # BF16 rounds to an infinity from 2^128 (1 - 2^-9) on; FP32's error is below 2^-16 of a result
        # (89 2^-23 of the sigmoid's), so nothing under 2^128 (1 - 2^-8) gets there, and none of the
        # results lie between that and 2^128
        finite = np.abs(want) < 2.0 ** 128 * (1 - 2.0 ** -8)
        assert (finite | (np.abs(want) >= 2.0 ** 128)).all()
        over = got.double().cpu().numpy()[~finite]
        assert (np.isinf(over) & (np.sign(over) == np.sign(want[~finite]))).all(), what
        close(torch.where(torch.from_numpy(finite), got.double().cpu(), 0.0),
              np.where(finite, want, 0.0), np.where(finite, tol, 0.0), what)
    return kept


def test_kept_values_past_fp32(m):
    """The largest BF16 numbers round up to 256 times the scale 2^120: a kept 2^128, which FP32 does
    not hold. Gates of that size, either sign, have gradients all the same."""
    top = bits_to_bf16(np.array([0x7F7F], np.uint16))[0].item()   # (2 - 2^-7) 2^127
    gates = torch.tensor([top, -top, 1.9375 * 2.0 ** 127, -1.9375 * 2.0 ** 127, 2.0 ** 127])
    x = torch.zeros(gates.numel(), 64)
    x[:, :32] = gates[:, None]
    x[:, 32:] = torch.linspace(-1, 1, 32)
    dh = (torch.linspace(-1, 1, 32) * 2.0 ** -8).expand(5, 32).contiguous().to(BF16)
    kept = check_backward(m, x.to(BF16), dh)
    assert (np.abs(kept[:4, :32]) == 2.0 ** 128).all()
    # and ups of that size, under gates of all sizes
    x = torch.zeros(5, 64)
    x[:, :32] = torch.tensor([-300.0, -80.0, -1.0, 0.0, 0.5])[:, None]
    x[:, 32:] = torch.where(torch.arange(32) % 2 == 0, top, -top)
    kept = check_backward(m, x.to(BF16), dh)
    assert (np.abs(kept[:, 32:]) == 2.0 ** 128).all()


@pytest.mark.parametrize("up,grad", [(2.0 ** 100, 2.0 ** 40), (2.0 ** 40, -2.0 ** 100),
                                     (-1.5 * 2.0 ** 126, 1.75 * 2.0 ** 70),
                                     (2.0 ** 127, 2.0 ** 3), (2.0 ** 90, 2.0 ** 30)])
def test_gradient_of_large_products(m, up, grad):
    """dh u past FP32's range, times the small factor of a gate far below zero."""
    gates = torch.tensor([-300.0, -100, -88, -80, -72, -64, -56, -48, -40, -30, -5, 4])
    x = torch.zeros(gates.numel(), 64)
    x[:, :32] = gates[:, None]
    x[:, 32:] = up
    dh = torch.full((gates.numel(), 32), grad).to(BF16)
    check_backward(m, x.to(BF16), dh)


@pytest.mark.parametrize("peak", [-126, -123, -121, -120, -119, -110, 0, 120])
def test_what_the_checkpoint_loses_by_block(m, peak):
    """Within 2^-4 of the value or 2^-17 of its block's largest, from blocks of 2^-120 on; below,
    where the scale is at its least, within 2^-4 or 2^-137."""
    g = torch.Generator().manual_seed(abs(peak))
    x = torch.randn(64, 256, generator=g, dtype=torch.float64).clamp(-1, 1)
    x *= 2.0 ** -torch.randint(0, 12, x.shape, generator=g).double()
    x[:, ::32] = 1 + 0.99 * torch.rand(64, 8, generator=g, dtype=torch.float64)
    x = (x * 2.0 ** peak).to(BF16)
    r = m.swiglu(x.to(DEV))
    kept, v = O.dequantize(u8(r.codes), u8(r.scales)), x.double().numpy()
    largest = np.abs(v).reshape(64, -1, 32).max(axis=2).repeat(32, axis=1)
    floor = np.where(largest >= 2.0 ** -120, 2.0 ** -17 * largest, 2.0 ** -137)
    assert (np.abs(kept - v) <= np.maximum(2.0 ** -4 * np.abs(v), floor)).all()
