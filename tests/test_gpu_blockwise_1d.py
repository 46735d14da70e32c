"""GPU parity of the 1 x 128 block-wise quantizer (both axes, and both from one read) and of
the 128 x 128 quantizer with a transposed copy: codes and scales bit for bit against the
oracle."""
import numpy as np
import pytest
import torch

import oracle.blockwise_oracle as B
import oracle.mxfp8_oracle as O
from tests.oracle_helpers import bits_to_bf16, gpu_ready, u8

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [O.BW_SCALE_FP32, O.BW_SCALE_POW2]


@pytest.fixture(scope="module")
def m():
    mod = gpu_ready()
    yield mod
    assert mod.device_status() == mod.OK


def rand_bits(g, shape):
    """Rows and columns of widely spread magnitude, some of them zero."""
    x = g.standard_normal(shape) * np.exp2(g.integers(-30, 30, size=(shape[0], 1)))
    x *= np.exp2(g.integers(-12, 12, size=(1, shape[1])))
    x[g.random(shape) < 0.1] = 0.0
    x[g.random(shape[0]) < 0.1] = 0.0
    f = x.astype(np.float32).view(np.uint32).astype(np.uint64)
    return ((f + 0x7FFF + ((f >> 16) & 1)) >> 16).astype(np.uint16)


def same(q, s, rq, rs):
    np.testing.assert_array_equal(u8(q), rq)
    np.testing.assert_array_equal(s.cpu().numpy().view(np.uint32), rs.view(np.uint32))


@pytest.mark.parametrize("shape", [(1, 16), (1, 4096), (7, 128), (37, 272), (128, 128),
                                   (129, 400), (200, 1040), (256, 144)])
@pytest.mark.parametrize("st", TYPES)
def test_both_axes_and_dual(m, shape, st):
    bits = rand_bits(np.random.default_rng(shape[0] * 7 + shape[1]), shape)
    x = bits_to_bf16(bits).to(DEV)
    want_r, want_c = B.quantize_1d(bits, B.ROW, st), B.quantize_1d(bits, B.COL, st)
    same(*m.quantize_blockwise_1d(x, m.ROW, st), *want_r)
    same(*m.quantize_blockwise_1d(x, m.COL, st), *want_c)
    rq, rs, cq, cs = m.quantize_blockwise_1d_dual(x, st)
    same(rq, rs, *want_r)
    same(cq, cs, *want_c)


@pytest.mark.parametrize("shape", [(5, 8), (130, 24), (17, 136)])
def test_transposed_copy_alone_takes_columns_in_eights(m, shape):
    bits = rand_bits(np.random.default_rng(shape[1]), shape)
    same(*m.quantize_blockwise_1d(bits_to_bf16(bits).to(DEV), m.COL), *B.quantize_1d(bits, B.COL))


@pytest.mark.parametrize("shape", [(16, 16), (128, 256), (144, 400), (272, 128)])
@pytest.mark.parametrize("st", TYPES)
def test_weight_and_its_transpose(m, shape, st):
    bits = rand_bits(np.random.default_rng(shape[0] + shape[1]), shape)
    q, s, qt, s_t = m.quantize_blockwise_dual(bits_to_bf16(bits).to(DEV), st)
    rq, rs = O.quantize_blockwise_2d(bits, st)
    same(q, s, rq, rs)
    same(qt, s_t, np.ascontiguousarray(rq.T), np.ascontiguousarray(rs.T))


@pytest.mark.parametrize("st", TYPES)
def test_nan_infinity_zero_and_tiny_blocks(m, st):
    x = np.zeros((200, 272), np.float32)
    x[3, 5], x[3, 6], x[3, 200] = np.nan, -1.0, 2.0
    x[130, 20], x[131, 20] = -np.inf, 3.0
    x[50, :] = -0.0
    x[60, :] = 1e-38
    x[61, 130] = 9.2e-41                       # a BF16 subnormal alone in its row block
    bits = (x.view(np.uint32) >> 16).astype(np.uint16)
    t = bits_to_bf16(bits).to(DEV)
    same(*m.quantize_blockwise_1d(t, m.ROW, st), *B.quantize_1d(bits, B.ROW, st))
    same(*m.quantize_blockwise_1d(t, m.COL, st), *B.quantize_1d(bits, B.COL, st))
    sq = bits[:192]
    q, s, qt, s_t = m.quantize_blockwise_dual(bits_to_bf16(sq).to(DEV), st)
    rq, rs = O.quantize_blockwise_2d(sq, st)
    same(q, s, rq, rs)
    same(qt, s_t, np.ascontiguousarray(rq.T), np.ascontiguousarray(rs.T))


@pytest.mark.parametrize("amax", [1.0, 448.0, 2.0 ** 100, 1.5 * 2.0 ** -120])
@pytest.mark.parametrize("st", TYPES)
def test_every_bf16_value_below_the_block_maximum(m, st, amax):
    allb = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    vals = O.bf16_to_f64(allb)
    top = np.float32(amax).view(np.uint32) >> 16
    keep = allb[np.isfinite(vals) & (np.abs(vals) <= amax)]
    rows = -(-keep.size // 127)
    bits = np.zeros((rows, 128), np.uint16)
    bits[:, 1:].reshape(-1)[...] = 0
    flat = np.zeros(rows * 127, np.uint16)
    flat[:keep.size] = keep
    bits[:, 1:] = flat.reshape(rows, 127)
    bits[:, 0] = top
    same(*m.quantize_blockwise_1d(bits_to_bf16(bits).to(DEV), m.ROW, st),
         *B.quantize_1d(bits, B.ROW, st))


def test_given_buffers_are_written_and_nothing_past_them(m):
    bits = rand_bits(np.random.default_rng(9), (37, 144))
    x = bits_to_bf16(bits).to(DEV)
    pad = 512
    big_q = torch.full((144 * 48 + pad,), 0xAB, dtype=torch.uint8, device=DEV)
    big_s = torch.full((144 + pad,), -7.0, dtype=torch.float32, device=DEV)
    m.quantize_blockwise_1d(x, m.COL, out=big_q, scale_inv=big_s)
    rq, rs = B.quantize_1d(bits, B.COL)
    np.testing.assert_array_equal(u8(big_q[:144 * 48]).reshape(144, 48), rq)
    np.testing.assert_array_equal(big_s[:144].cpu().numpy(), rs[0])
    assert (big_q[144 * 48:] == 0xAB).all() and (big_s[144:] == -7.0).all()


def test_empty_inputs(m):
    x = torch.empty((0, 128), dtype=torch.bfloat16, device=DEV)
    q, s = m.quantize_blockwise_1d(x, m.ROW)
    assert q.shape == (0, 128) and s.shape == (1, 0)
    q, s = m.quantize_blockwise_1d(x, m.COL)
    assert q.shape == (128, 0) and s.shape == (0, 128)


def test_refusals(m):
    x = torch.zeros((32, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        m.quantize_blockwise_1d(x.float())
    with pytest.raises(ValueError):
        m.quantize_blockwise_1d(x.t())
    with pytest.raises(ValueError):
        m.quantize_blockwise_1d(x, axis=2)
    with pytest.raises(ValueError):
        m.quantize_blockwise_1d(x, out=torch.empty(10, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        m.quantize_blockwise_1d_dual(x, col_scale_inv=torch.empty(3, device=DEV))
    with pytest.raises(m.MXFP8Error) as e:
        m.quantize_blockwise_1d(x, scale_type=5)
    assert e.value.status == m.ERR_INVALID_ARG
    for call, shape in ((m.quantize_blockwise_1d, (32, 24)), (m.quantize_blockwise_dual, (24, 32)),
                        (m.quantize_blockwise_1d_dual, (32, 40))):
        with pytest.raises(m.MXFP8Error) as e:
            call(torch.zeros(shape, dtype=torch.bfloat16, device=DEV))
        assert e.value.status == m.ERR_ALIGNMENT


def test_input_past_2_to_the_31_elements(m):
    rows, cols = 65544, 32784
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(5)
    for i in range(0, rows, 8193):
        x[i:i + 8193] = torch.randn((min(8193, rows - i), cols), generator=g, device=DEV)
    bits = x.view(torch.int16)
    ri, ci = [0, 4096, 65535, 65536, rows - 1], [0, 777, 32767, 32768, cols - 1]
    rb = bits[ri].cpu().numpy().view(np.uint16)
    cb = bits[:, ci].cpu().numpy().view(np.uint16)
    rq, rs, cq, cs = m.quantize_blockwise_1d_dual(x, O.BW_SCALE_FP32)
    same(rq[ri], rs[:, ri], *B.quantize_1d(rb, B.ROW, O.BW_SCALE_FP32))
    same(cq[ci], cs[:, ci], *B.quantize_1d(np.ascontiguousarray(cb), B.COL, O.BW_SCALE_FP32))
