"""CPU oracle of the 1 x 128 block-wise quantizer and of the block-wise GEMM (numpy, float64).

Test infrastructure only: it shares no code with the GPU path. Codes and scales follow the
rule of the 128 x 128 block-wise quantizer (oracle.mxfp8_oracle.quantize_blockwise_2d),
applied to blocks of 128 along one axis ("End-to-End MXFP8 RL on Blackwell", section "A
different grid, and drift").
"""
import numpy as np

from oracle.mxfp8_oracle import (BW_SCALE_FP32, E4M3_MAX, E4M3_NAN, RULE_CEIL, bf16_to_f64,
                                 block_scale_exponent, e4m3_decode, e4m3_round_code)

BLOCK = 128
ROW, COL = 0, 1


def factor(amax, scale_type):
    """The single-precision factor of a finite block."""
    if amax == 0.0:
        return np.float32(1.0)
    if scale_type == BW_SCALE_FP32:
        with np.errstate(over="ignore"):
            s = np.float32(E4M3_MAX) / np.float32(amax)
        return s if np.isfinite(s) else np.finfo(np.float32).max
    return np.float32(np.ldexp(1.0, -int(block_scale_exponent(amax, RULE_CEIL))))


def quantize_1d(x_bits, axis=ROW, scale_type=BW_SCALE_FP32):
    """(codes, scale_inv) as mxfp8_quantize_blockwise_1d writes them: ROW: [rows, cols] and
    [ceil(cols/128), rows]; COL: [cols, rows rounded up to 16] and [ceil(rows/128), cols]."""
    x = bf16_to_f64(x_bits)
    if axis == COL:
        x = x.T
    r, n = x.shape
    nb = -(-n // BLOCK)
    codes = np.zeros((r, n if axis == ROW else -(-n // 16) * 16), np.uint8)
    inv = np.empty((nb, r), np.float32)
    for b in range(nb):
        for i in range(r):
            blk = x[i, b * BLOCK:(b + 1) * BLOCK]
            out = codes[i, b * BLOCK:min((b + 1) * BLOCK, n)]
            if not np.all(np.isfinite(blk)):
                out[...] = E4M3_NAN | (np.signbit(blk).astype(np.int64) << 7)
                inv[b, i] = np.nan
                continue
            s = factor(float(np.max(np.abs(blk))), scale_type)
            out[...] = e4m3_round_code((blk.astype(np.float32) * s).astype(np.float64))
            inv[b, i] = np.float32(1.0) / s
    return codes, inv


def dequantize_1d(codes, inv):
    """[r, n] codes with scale inverses [blocks, r], in float64."""
    v = e4m3_decode(codes)
    return v * np.repeat(inv.astype(np.float64).T, BLOCK, axis=1)[:, :v.shape[1]]


def dequantize_2d(codes, inv):
    v = e4m3_decode(codes)
    s = np.repeat(np.repeat(inv.astype(np.float64), BLOCK, axis=0), BLOCK, axis=1)
    return v * s[:v.shape[0], :v.shape[1]]


def gemm_bound(abs_sum, k):
    """Error bound of the FP32 result: a 128-deep block is accumulated by the tensor cores,
    each of its 128 additions losing at most 2^-23 of the running magnitude; every block is
    then scaled (two roundings) and added (one, and one for each later block) in FP32."""
    nkb = -(-k // BLOCK)
    return abs_sum * (BLOCK * 2.0 ** -23 + (nkb + 3) * 2.0 ** -24)
