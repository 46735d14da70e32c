"""GPU parity of the gated activation, its 8-bit checkpoint and the gradient from it.

Codes and scale bytes match the oracle's quantizer bit for bit. h, dg and du are FP32 results
(oracle/swiglu_oracle.py derives how far those may be off) rounded to BF16: half a step more,
2^-8 of the result, or 2^-134 among subnormals."""
import numpy as np
import pytest
import torch

import oracle.mxfp8_oracle as O
import oracle.swiglu_oracle as S
from tests.oracle_helpers import bf16_bits, gpu_ready, u8

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
SHAPES = [(1, 32), (1, 12288), (3, 64), (37, 96), (129, 768), (1021, 160), (70, 4128), (8, 2048)]


@pytest.fixture(scope="module")
def m():
    mod = gpu_ready()
    yield mod
    assert mod.device_status() == mod.OK


def inputs(seed, rows, width):
    """[rows, 2 width] with gates over all of the sigmoid's range, small and large ups."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, 2 * width, generator=g)
    x[:, :width] *= torch.exp2(torch.randint(-6, 6, (rows, width), generator=g).float())
    x[:, width + 1::7] *= 30
    return x.to(BF16)


def close(got, want, tol, what):
    got = got.double().cpu().numpy()
    err, tol = np.abs(got - want), tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want) + 2.0 ** -134
    assert (err <= tol).all(), (what, np.max(err - tol))


def check_forward(m, x, rule=1, **kw):
    width = x.shape[1] // 2
    r = m.swiglu(x.to(DEV), rule=rule, **kw)
    codes, scales = O.quantize(bf16_bits(x), O.ROW, rule=rule)
    np.testing.assert_array_equal(u8(r.codes), codes)
    np.testing.assert_array_equal(u8(r.scales), scales)
    v = x.double().numpy()
    g, u = v[:, :width], v[:, width:]
    close(r.h, S.forward(g, u), S.forward_error(g, u), "h")
    bare = m.swiglu(x.to(DEV), checkpoint=False)
    assert bare.codes is None and bare.scales is None and torch.equal(bare.h, r.h)
    return r


@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("rows,width", SHAPES)
def test_forward(m, rows, width, rule):
    check_forward(m, inputs(rows, rows, width), rule)


@pytest.mark.parametrize("rows,width", SHAPES)
def test_backward(m, rows, width):
    x = inputs(rows + 1, rows, width)
    r = m.swiglu(x.to(DEV))
    g = torch.Generator().manual_seed(rows)
    dh = torch.randn(rows, width, generator=g).to(BF16)
    grad, h = m.swiglu_backward(dh.to(DEV), r.codes, r.scales, recompute=True)
    kept = O.dequantize(u8(r.codes), u8(r.scales))
    a, u, d = kept[:, :width], kept[:, width:], dh.double().numpy()
    dg, du = S.backward(a, u, d)
    eg, eu = S.backward_error(a, u, d)
    close(grad[:, :width], dg, eg, "dg")
    close(grad[:, width:], du, eu, "du")
    close(h, S.forward(a, u), S.forward_error(a, u), "h")
    alone, none = m.swiglu_backward(dh.to(DEV), r.codes, r.scales)
    assert none is None and torch.equal(alone, grad)
    dhd = dh.to(DEV)      # h in place of the gradient it came with
    again, same = m.swiglu_backward(dhd, r.codes, r.scales, recompute=True, out_h=dhd)
    assert same is dhd and torch.equal(again, grad) and torch.equal(dhd, h)


def test_checkpoint_is_the_quantizers(m):
    x = inputs(5, 333, 1024).to(DEV)
    for rule in (m.RULE_FLOOR, m.RULE_CEIL):
        r = m.swiglu(x, rule=rule)
        codes, scales = m.quantize(x, m.ROW, m.LINEAR, rule=rule)
        assert torch.equal(r.codes, codes) and torch.equal(r.scales.view(-1), scales.view(-1))


def test_what_the_checkpoint_loses(m):
    """With the round-up rule nothing saturates: a kept value is within 2^-4 of itself or 2^-17 of
    its block's largest."""
    x = inputs(6, 64, 512)
    r = m.swiglu(x.to(DEV))
    kept, v = O.dequantize(u8(r.codes), u8(r.scales)), x.double().numpy()
    peak = np.abs(v).reshape(64, -1, 32).max(axis=2).repeat(32, axis=1)
    assert (np.abs(kept - v) <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -17 * peak)).all()


def test_nan_and_infinity(m):
    x = inputs(7, 8, 64)
    x[1, 3], x[2, 70], x[3, 40], x[4, 2] = float("nan"), float("nan"), float("inf"), -float("inf")
    x[5, 100] = float("inf")
    r = m.swiglu(x.to(DEV))
    codes, scales = O.quantize(bf16_bits(x), O.ROW, rule=1)
    np.testing.assert_array_equal(u8(r.codes), codes)
    np.testing.assert_array_equal(u8(r.scales), scales)
    h = r.h.float().cpu()
    assert h[1, 3].isnan() and h[2, 6].isnan() and h[4, 2].isnan()
    assert h[3, 40].isinf() and h[5, 36].isinf()
    ok = torch.ones_like(h, dtype=torch.bool)
    for row, col in ((1, 3), (2, 6), (3, 40), (4, 2), (5, 36)):
        ok[row, col] = False
    assert h[ok].isfinite().all()
    grad, again = m.swiglu_backward(torch.ones(8, 64, dtype=BF16, device=DEV), r.codes, r.scales,
                                    recompute=True)
    grad, again = grad.float().cpu(), again.float().cpu()
    assert grad[1, :32].isnan().all() and grad[1, 64:96].isnan().all()   # the block's gate
    assert grad[1, 32:64].isfinite().all() and again[1, 32:].isfinite().all()
    assert grad[2, :32].isnan().all() and grad[2, 64:96].isfinite().all()   # the block's up
    assert grad[0].isfinite().all() and grad[6:].isfinite().all()


def test_far_gates(m):
    """Sigmoids at the ends of FP32's range."""
    gates = torch.tensor([-3e38, -1e4, -200, -104, -95, -89, -88, -87, -60, -20, -1e-3, -1e-39, 0.0,
                          1e-39, 1e-3, 20, 60, 88, 200, 1e4, 3e38]).to(BF16)
    x = torch.zeros(gates.numel(), 64)
    x[:, :32] = gates.float()[:, None]
    x[:, 32:] = torch.linspace(-1, 1, 32)   # 3e38 of them is still a BF16 value
    check_forward(m, x.to(BF16))
    dh = torch.linspace(0.1, 1, 32).expand(gates.numel(), 32).contiguous().to(BF16)
    r = m.swiglu(x.to(BF16).to(DEV))
    grad, _ = m.swiglu_backward(dh.to(DEV), r.codes, r.scales)
    kept = O.dequantize(u8(r.codes), u8(r.scales))
    d = dh.double().numpy()
    dg, du = S.backward(kept[:, :32], kept[:, 32:], d)
    eg, eu = S.backward_error(kept[:, :32], kept[:, 32:], d)
    close(grad[:, :32], dg, eg, "dg")
    close(grad[:, 32:], du, eu, "du")


def test_buffers_on_16_bytes(m):
    """Tensors that start on 16 but not on 32 bytes, margins untouched."""
    rows, width = 33, 96
    x = inputs(8, rows, width)

    def odd(n, dtype):
        size = torch.empty(0, dtype=dtype).element_size()
        raw = torch.full((n * size + 96,), 0x5B, dtype=torch.uint8, device=DEV)
        part = raw[16:16 + n * size]
        return part.view(dtype), raw, slice(16 + n * size, None)

    xs, _, _ = odd(rows * 2 * width, BF16)
    xs.copy_(x.view(-1))
    h, h_raw, h_end = odd(rows * width, BF16)
    codes, c_raw, c_end = odd(rows * 2 * width, torch.uint8)
    scales, s_raw, s_end = odd(rows * width // 16, torch.uint8)
    r = check_forward(m, x)
    m.swiglu(xs.view(rows, 2 * width), out=h, codes=codes, scales=scales)
    assert torch.equal(h.view(rows, width), r.h)
    assert torch.equal(codes.view(rows, -1), r.codes)
    assert torch.equal(scales.view(rows, -1), r.scales)
    dh = torch.randn(rows, width, generator=torch.Generator().manual_seed(1)).to(BF16).to(DEV)
    want, want_h = m.swiglu_backward(dh, r.codes, r.scales, recompute=True)
    grad, g_raw, g_end = odd(rows * 2 * width, BF16)
    m.swiglu_backward(dh, codes, scales, recompute=True, out=grad, out_h=h)
    assert torch.equal(grad.view(rows, -1), want) and torch.equal(h.view(rows, -1), want_h)
    for raw, end in ((h_raw, h_end), (c_raw, c_end), (s_raw, s_end), (g_raw, g_end)):
        assert (raw[end] == 0x5B).all() and (raw[:16] == 0x5B).all()


def test_empty(m):
    for shape in ((0, 64), (5, 0)):
        r = m.swiglu(torch.empty(shape, dtype=BF16, device=DEV))
        assert r.h.shape == (shape[0], shape[1] // 2)
        grad, h = m.swiglu_backward(r.h, r.codes, r.scales, recompute=True)
        assert grad.shape == shape and h.shape == r.h.shape


def test_captured_and_on_another_stream(m):
    x = inputs(9, 257, 256).to(DEV)
    dh = torch.randn(257, 256, device=DEV).to(BF16)

    def step(stream=None):
        r = m.swiglu(x, stream=stream)
        return (*r, *m.swiglu_backward(dh, r.codes, r.scales, recompute=True, stream=stream))

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held = step()
    x.copy_(inputs(10, 257, 256))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(held, step()):
        assert torch.equal(a, b)


def test_past_two_to_the_31_elements(m):
    rows, width = 66000, 16512
    x = torch.zeros(rows, 2 * width, dtype=BF16, device=DEV)
    x[:, width - 32:width] = 3.0
    x[:, -32:] = (torch.arange(rows, device=DEV) % 13).to(BF16)[:, None]
    assert x.numel() > 2 ** 31
    r = m.swiglu(x)
    small = m.swiglu(torch.cat([x[:, width - 32:width], x[:, -32:]], dim=1).contiguous())
    assert torch.equal(r.h[:, -32:], small.h) and not r.h[:, :-32].any()
    assert torch.equal(r.codes[:, -32:], small.codes[:, 32:])
    assert torch.equal(r.scales[:, -1], small.scales[:, 1])
    dh = torch.ones(rows, width, dtype=BF16, device=DEV)
    grad, h = m.swiglu_backward(dh, r.codes, r.scales, recompute=True)
    want, want_h = m.swiglu_backward(dh[:, :32].contiguous(), small.codes, small.scales,
                                     recompute=True)
    assert torch.equal(grad[:, width - 32:width], want[:, :32])
    assert torch.equal(grad[:, -32:], want[:, 32:]) and torch.equal(h[:, -32:], want_h)
