"""GPU parity of the block-wise FP8 GEMM against the float64 oracle, in all three
directions, with a bound derived from FP32 accumulation (oracle.blockwise_oracle)."""
import numpy as np
import pytest
import torch

import oracle.blockwise_oracle as B
import oracle.mxfp8_oracle as O
from tests.oracle_helpers import gpu_ready

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def m():
    mod = gpu_ready()
    yield mod
    assert mod.device_status() == mod.OK


def codes(g, r, n):
    """Random finite E4M3 codes of every magnitude."""
    c = g.integers(0, 256, size=(r, n)).astype(np.uint8)
    return np.where((c & 0x7F) == 0x7F, c & 0x80, c).astype(np.uint8)


def operands(seed, mm, n, k, wgrad, spread=6):
    g = np.random.default_rng(seed)
    kb = -(-k // 128)
    scale = lambda *shape: (g.random(shape) + 0.5).astype(np.float32) * \
        np.exp2(g.integers(-spread, spread + 1, size=shape)).astype(np.float32)  # noqa: E731
    a, sa = codes(g, mm, k), scale(kb, mm)
    b = codes(g, n, k)
    sb = scale(kb, n) if wgrad else scale(-(-n // 128), kb)
    return a, sa, b, sb


def reference(a, sa, b, sb, wgrad):
    da = B.dequantize_1d(a, sa)
    db = B.dequantize_1d(b, sb) if wgrad else B.dequantize_2d(b, sb)
    return da @ db.T, np.abs(da) @ np.abs(db).T


def check(got, ref, ab, k, bf16):
    bound = B.gemm_bound(ab, k)
    if bf16:
        bound = bound + np.abs(ref) * 2.0 ** -8 + 2.0 ** -133
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err <= bound), f"{np.sum(~(err <= bound))} outside, worst {np.max(err / bound)}"


def to(*arrays):
    return [torch.from_numpy(x).to(DEV) for x in arrays]


SIZES = [(1, 128, 128), (1, 8, 16), (3, 264, 400), (16, 128, 1024), (17, 384, 640),
         (33, 1032, 272), (64, 512, 2048), (65, 136, 144), (127, 256, 4096), (128, 128, 256),
         (129, 136, 528), (200, 648, 1168), (300, 1024, 512), (513, 264, 784)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("fp32", [False, True])
def test_forward(m, size, fp32):
    mm, n, k = size
    ops = operands(mm + n + k, mm, n, k, False)
    a, sa, b, sb = to(*ops)
    c = m.blockwise_gemm(a, sa, b, sb, m.FPROP, m.OUT_FP32 if fp32 else m.OUT_BF16)
    check(c, *reference(*ops, False), k, not fp32)


@pytest.mark.parametrize("size", [(8, 8, 16), (128, 128, 128), (136, 264, 48), (264, 520, 1040),
                                  (1, 128, 256), (768, 1024, 208), (41, 72, 2000)])
@pytest.mark.parametrize("fp32", [False, True])
def test_weight_gradient(m, size, fp32):
    mm, n, k = size
    ops = operands(mm + n + k, mm, n, k, True)
    a, sa, b, sb = to(*ops)
    c = m.blockwise_gemm(a, sa, b, sb, m.WGRAD, m.OUT_FP32 if fp32 else m.OUT_BF16)
    check(c, *reference(*ops, True), k, not fp32)


def gpu_reference(a, sa, b, sb, wgrad):
    """The same in float64 on the GPU, for sizes that take long on the CPU."""
    def deq(q, s):
        return q.view(torch.float8_e4m3fn).double() * s.double()[:, :q.shape[1]]
    da = deq(a, sa.t().repeat_interleave(128, 1))
    db = deq(b, sb.t().repeat_interleave(128, 1)) if wgrad else \
        deq(b, sb.repeat_interleave(128, 0).repeat_interleave(128, 1)[:b.shape[0]])
    return (da @ db.t()).cpu().numpy(), (da.abs() @ db.abs().t()).cpu().numpy()


@pytest.mark.parametrize("size,wgrad", [((2048, 2056, 528), False), ((1999, 2304, 1040), False),
                                        ((2056, 1928, 656), True), ((4096, 4096, 256), False),
                                        ((1280, 5000, 144), True), ((700, 8200, 384), False)])
@pytest.mark.parametrize("fp32", [False, True])
def test_many_tiles(m, size, wgrad, fp32):
    mm, n, k = size
    a, sa, b, sb = to(*operands(mm + n, mm, n, k, wgrad))
    c = m.blockwise_gemm(a, sa, b, sb, m.WGRAD if wgrad else m.FPROP,
                         m.OUT_FP32 if fp32 else m.OUT_BF16)
    check(c, *gpu_reference(a, sa, b, sb, wgrad), k, not fp32)


@pytest.mark.parametrize("mm", [1, 20, 100, 300, 2304])
def test_scales_of_extreme_magnitude(m, mm):
    """Pairs of block scales whose product leaves the normal range, while the scaled sums
    stay inside it."""
    n, k = 2304 if mm == 2304 else 264, 512
    a, sa, b, sb = operands(mm, mm, n, k, False, spread=0)
    sa[0], sb[:, 0] = sa[0] * np.float32(2.0 ** -90), sb[:, 0] * np.float32(2.0 ** -46)
    sa[1], sb[:, 1] = sa[1] * np.float32(2.0 ** 120), sb[:, 1] * np.float32(2.0 ** -140)
    sa[2], sb[:, 2] = sa[2] * np.float32(2.0 ** -126), sb[:, 2] * np.float32(2.0 ** 100)
    sa[3], sb[:, 3] = sa[3] * np.float32(2.0 ** -80), sb[:, 3] * np.float32(2.0 ** -50)
    da, db = B.dequantize_1d(a, sa), B.dequantize_2d(b, sb)
    got = m.blockwise_gemm(*to(a, sa, b, sb), m.FPROP, m.OUT_FP32)
    # FP32 keeps subnormals: the bound gains one such rounding a block
    bound = B.gemm_bound(np.abs(da) @ np.abs(db).T, k) + 8 * 2.0 ** -149
    err = np.abs(got.double().cpu().numpy() - da @ db.T)
    assert np.all(err <= bound), np.max(err / bound)


@pytest.mark.parametrize("mm", [2, 40, 260, 2304])
def test_nan_blocks_reach_their_rows_and_columns_only(m, mm):
    n, k = 2304 if mm == 2304 else 392, 384
    a, sa, b, sb = operands(5, mm, n, k, False)
    a[1, 130:256], sa[1, 1] = 0x7F, np.nan
    got = m.blockwise_gemm(*to(a, sa, b, sb)).float().cpu().numpy()
    assert np.isnan(got[1]).all() and not np.isnan(np.delete(got, 1, axis=0)).any()
    a, sa, b, sb = operands(6, mm, n, k, False)
    b[128:256, 256:384], sb[1, 2] = 0x7F, np.nan
    got = m.blockwise_gemm(*to(a, sa, b, sb)).float().cpu().numpy()
    assert np.isnan(got[:, 128:256]).all()
    assert not np.isnan(got[:, :128]).any() and not np.isnan(got[:, 256:]).any()


@pytest.mark.parametrize("mm,n,k", [(1, 256, 1024), (48, 520, 656), (300, 264, 528),
                                    (2304, 2312, 272)])
def test_same_bytes_every_time_and_nothing_outside_the_output(m, mm, n, k):
    a, sa, b, sb = to(*operands(1, mm, n, k, False))
    first = m.blockwise_gemm(a, sa, b, sb)
    guard = torch.full((mm * n + 1024,), 3.0, dtype=torch.bfloat16, device=DEV)
    for _ in range(3):
        m.blockwise_gemm(a, sa, b, sb, out=guard)
        assert torch.equal(guard[:mm * n].view(mm, n), first)
    assert (guard[mm * n:] == 3.0).all()


def test_from_the_quantizers(m):
    """Forward, data gradient and weight gradient of one layer for an odd number of tokens,
    each operand from its quantizer, against the oracle on the dequantized operands."""
    g = torch.Generator().manual_seed(3)
    t, n, k = 203, 272, 400
    x = torch.randn(t, k, generator=g).to(torch.bfloat16).to(DEV)
    w = (torch.randn(n, k, generator=g) * 0.02).to(torch.bfloat16).to(DEV)
    dy = torch.randn(t, n, generator=g).to(torch.bfloat16).to(DEV)
    xq, xs, xt, xts = m.quantize_blockwise_1d_dual(x, m.BW_POW2)
    wq, ws, wt, wts = m.quantize_blockwise_dual(w, m.BW_POW2)
    dq, ds, dt, dts = m.quantize_blockwise_1d_dual(dy, m.BW_POW2)
    num = lambda *ts: [v.cpu().numpy() for v in ts]  # noqa: E731
    y = m.blockwise_gemm(xq, xs, wq, ws, m.FPROP, m.OUT_FP32)
    check(y, *reference(*num(xq, xs, wq, ws), False), k, False)
    dx = m.blockwise_gemm(dq, ds, wt, wts, m.DGRAD, m.OUT_FP32)
    check(dx, *reference(*num(dq, ds, wt, wts), False), n, False)
    dw = m.blockwise_gemm(dt, dts, xt, xts, m.WGRAD, m.OUT_FP32)
    check(dw, *reference(*num(dt, dts, xt, xts), True), t, False)
    # quantization error alone: within 2^-4 of each operand's block maximum per factor
    exact = x.double() @ w.double().t()
    assert (y.double() - exact).norm() < 0.06 * exact.norm()


def test_empty_sizes(m):
    e8 = lambda *s: torch.empty(s, dtype=torch.uint8, device=DEV)  # noqa: E731
    f = lambda *s: torch.empty(s, dtype=torch.float32, device=DEV)  # noqa: E731
    assert m.blockwise_gemm(e8(0, 128), f(1, 0), e8(64, 128), f(1, 1)).shape == (0, 64)
    assert m.blockwise_gemm(e8(5, 128), f(1, 5), e8(0, 128), f(0, 1)).shape == (5, 0)
    c = m.blockwise_gemm(e8(5, 0), f(0, 5), e8(64, 0), f(1, 0), m.WGRAD, m.OUT_FP32)
    assert c.shape == (5, 64) and (c == 0).all()


def test_refusals(m):
    a, sa, b, sb = to(*operands(1, 4, 128, 256, False))
    with pytest.raises(ValueError):
        m.blockwise_gemm(a, sa, b[:, :128].contiguous(), sb)
    with pytest.raises(ValueError):
        m.blockwise_gemm(a.float(), sa, b, sb)
    with pytest.raises(ValueError):
        m.blockwise_gemm(a, sa[:1].contiguous(), b, sb)
    with pytest.raises(ValueError):
        m.blockwise_gemm(a, sa, b, sb[:, :1].contiguous())
    with pytest.raises(ValueError):
        m.blockwise_gemm(a, sa, b, sb, m.WGRAD)      # a scale per column and block is needed
    with pytest.raises(ValueError):
        m.blockwise_gemm(a, sa.double(), b, sb)
    with pytest.raises(ValueError):
        m.blockwise_gemm(a, sa, b, sb, out=torch.empty(7, dtype=torch.bfloat16, device=DEV))
    for bad in ((a, sa, b, sb, 7), (a, sa, b, sb, m.FPROP, 9)):
        with pytest.raises((m.MXFP8Error, ValueError)):
            m.blockwise_gemm(*bad)
    a, sa, b, sb = to(*operands(1, 4, 132, 256, False))
    with pytest.raises(m.MXFP8Error) as e:
        m.blockwise_gemm(a, sa, b, sb)
    assert e.value.status == m.ERR_ALIGNMENT


def test_other_stream_and_graph(m):
    a, sa, b, sb = to(*operands(2, 70, 640, 512, False))
    want = m.blockwise_gemm(a, sa, b, sb)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = m.blockwise_gemm(a, sa, b, sb, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        m.blockwise_gemm(a, sa, b, sb, out=out)
    for _ in range(2):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)


@pytest.mark.parametrize("mm,n", [(5, 2048), (300, 512), (2304, 2304)])
def test_wait_limit_is_reported_and_the_next_call_works(m, mm, n):
    """A pipeline wait limit far below a tile's time: the call latches a timeout, leaves
    nothing behind, and the same call is right again with the default limit."""
    a, sa, b, sb = to(*operands(3, mm, n, 2048, False))
    want = m.blockwise_gemm(a, sa, b, sb)
    torch.cuda.synchronize()
    m.set_wait_limit_ns(1)
    try:
        m.blockwise_gemm(a, sa, b, sb)
        assert m.device_status() in (m.ERR_TIMEOUT, m.OK)
    finally:
        m.set_wait_limit_ns(0)
    assert torch.equal(m.blockwise_gemm(a, sa, b, sb), want)
    assert m.device_status() == m.OK


@pytest.mark.parametrize("wgrad,fp32,pow2", [(False, False, False), (True, True, False),
                                             (True, True, True)])
def test_output_past_2_to_the_31_elements(m, wgrad, fp32, pow2):
    mm, n, k = 65544, 32776, 128
    a, sa, b, sb = operands(21, mm, n, k, wgrad)
    if pow2:
        sa, sb = np.exp2(np.floor(np.log2(sa))), np.exp2(np.floor(np.log2(sb)))
    c = m.blockwise_gemm(*to(a, sa, b, sb), m.WGRAD if wgrad else m.FPROP,
                         m.OUT_FP32 if fp32 else m.OUT_BF16)
    ri = np.array([0, 1, 32767, 65409, 65535, 65536, mm - 1])
    ci = np.array([0, 7, 16384, 32767, 32768, n - 1])
    da = B.dequantize_1d(a[ri], sa[:, ri])
    db = B.dequantize_1d(b[ci], sb[:, ci]) if wgrad else \
        B.dequantize_1d(b[ci], sb[ci // 128].T)
    got = c[torch.from_numpy(ri).to(DEV)][:, torch.from_numpy(ci).to(DEV)]
    check(got, da @ db.T, np.abs(da) @ np.abs(db).T, k, not fp32)
