"""GB300-native MXFP8 quantizer and block-scaled GEMMs - Python binding.

Argument marshalling only: every call goes through the C ABI of ``libmxfp8.so``
(``include/mxfp8.h``), whose kernels do all of the work on the GPU. PyTorch provides
device memory and the current CUDA stream. There is no CPU fallback: if the library is
not built, or the device is not sm_103a, calls raise.

Method: "End-to-End MXFP8 RL on Blackwell" (verl blog post), section "The pipeline"
(paragraph "The format" and the learner and weight-synchronization paragraphs).
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional

import torch

ROW, COL = 0, 1
LINEAR, SWIZZLED = 0, 1
FPROP, DGRAD, WGRAD = 0, 1, 2
RULE_FLOOR, RULE_CEIL = 0, 1
OUT_BF16, OUT_FP32 = 0, 1

OK, ERR_INVALID_ARG, ERR_ALIGNMENT, ERR_UNSUPPORTED_ARCH, ERR_CUDA, ERR_BAD_OFFSETS, \
    ERR_TIMEOUT, ERR_BAD_TARGET, ERR_BAD_EXPERT = range(9)

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmxfp8.so")

# every symbol include/mxfp8.h declares: (name, restype, argtypes)
_P, _I64, _I, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
_D = ctypes.c_double
SIGNATURES = {
    "mxfp8_version": (_I, []),
    "mxfp8_status_string": (ctypes.c_char_p, [_I]),
    "mxfp8_scale_bytes": (_SZ, [_I64, _I64, _I, _I]),
    "mxfp8_grouped_scale_bytes": (_SZ, [_I64, _I64, _I, _I]),
    "mxfp8_quantize": (_I, [_P, _I64, _I64, _I, _P, _P, _I, _P]),
    "mxfp8_quantize_rule": (_I, [_P, _I64, _I64, _I, _P, _P, _I, _I, _P]),
    "mxfp8_quantize_dual": (_I, [_P, _I64, _I64, _P, _P, _P, _P, _I, _P]),
    "mxfp8_quantize_dual_multi": (_I, [_P, _I, _I, _P]),
    "mxfp8_blockwise_scale_count": (_SZ, [_I64, _I64]),
    "mxfp8_quantize_blockwise": (_I, [_P, _I64, _I64, _P, _P, _I, _P]),
    "mxfp8_quantize_blockwise_1d": (_I, [_P, _I64, _I64, _I, _P, _P, _I, _P]),
    "mxfp8_quantize_blockwise_1d_dual": (_I, [_P, _I64, _I64, _P, _P, _P, _P, _I, _P]),
    "mxfp8_quantize_blockwise_dual": (_I, [_P, _I64, _I64, _P, _P, _P, _P, _I, _P]),
    "mxfp8_quantize_batched": (_I, [_P, _I64, _I64, _I64, _I, _P, _P, _I, _P]),
    "mxfp8_quantize_grouped_dual": (_I, [_P, _I64, _I64, _P, _I, _P, _P, _P, _P, _P]),
    "mxfp8_quantize_grouped": (_I, [_P, _I64, _I64, _I, _P, _I, _P, _P, _P]),
    "mxfp8_gemm": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _I, _P]),
    "mxfp8_gemm_ws": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _I, _P, _SZ, _P]),
    "mxfp8_gemm_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I, _I]),
    "mxfp8_grouped_gemm": (_I, [_P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _I, _I, _P]),
    "mxfp8_blockwise_gemm": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _I, _P]),
    "mxfp8_blockwise_gemm_ws": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _I, _P, _SZ, _P]),
    "mxfp8_blockwise_gemm_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I]),
    "mxfp8_token_logprobs": (_I, [_P, _I, _I64, _I64, _I64, _P, _D, _P, _P, _P, _I, _P, _P, _P]),
    "mxfp8_token_logprobs_backward": (_I, [_P, _I, _I64, _I64, _I64, _P, _D, _P, _P, _P, _P, _I,
                                           _P, _P, _P, _I64, _P]),
    "mxfp8_route_rows": (_I64, [_I64, _I, _I]),
    "mxfp8_route": (_I, [_P, _I64, _I, _I, _I64, _P, _P, _P, _P]),
    "mxfp8_dispatch": (_I, [_P, _I, _I64, _I64, _I, _P, _P, _P, _I64, _P, _P]),
    "mxfp8_quantize_dispatch": (_I, [_P, _I64, _I64, _I, _P, _P, _P, _I64, _P, _I, _P, _P, _P,
                                     _P, _P]),
    "mxfp8_combine": (_I, [_P, _I, _I64, _I64, _I64, _I, _P, _P, _P, _P]),
    "mxfp8_combine_backward": (_I, [_P, _P, _I, _I64, _I64, _I, _P, _P, _P, _I64, _P, _P, _P]),
    "mxfp8_swiglu": (_I, [_P, _I64, _I64, _P, _P, _P, _I, _P]),
    "mxfp8_swiglu_backward": (_I, [_P, _P, _P, _I64, _I64, _P, _P, _P]),
    "mxfp8_selfcheck_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "mxfp8_selfcheck": (_I, [_P, _P, _P, _P, _I64, _I64, _P, _I64, _P, _SZ, _P, _P]),
    "mxfp8_selfcheck_noalloc": (_I, [_P, _P, _P, _P, _I64, _I64, _P, _I64, _P, _P]),
    "mxfp8_set_wait_limit_ns": (_I, [ctypes.c_uint64]),
    "mxfp8_get_device_status": (_I, [_P]),
}

_lib = None


class MXFP8Error(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        msg = lib().mxfp8_status_string(status).decode()
        super().__init__(f"{what}: {msg} (status {status})" if what else msg)


def lib() -> ctypes.CDLL:
    """The loaded C-ABI library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -c \"import __graft_entry__ as g; "
                "g.build()\"` (nvcc, sm_103a). There is no CPU fallback.")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def _check(status: int, what: str):
    if status != OK:
        raise MXFP8Error(status, what)


# The current stream's handle and the current device, asked for directly: building the stream's
# Python object takes 2.9 us on the GB300's host, as long as the launch itself. The direct names
# are torch's own, and a version without them takes the public way.
try:
    from torch._C import _cuda_getCurrentRawStream as _raw_stream, _cuda_getDevice as _device
except ImportError:
    _device = torch.cuda.current_device

    def _raw_stream(device):
        return torch.cuda.current_stream(device).cuda_stream


def _stream(stream=None):
    """A stream's handle."""
    if stream is None:
        return _raw_stream(torch.cuda.current_device())
    return stream.cuda_stream


def _ptr(t: torch.Tensor):
    return t.data_ptr()


def _require(t: torch.Tensor, dtype, name: str):
    """A tensor handed to the library: CUDA, of this dtype, contiguous, and on the current
    device (the library runs every call on the current device)."""
    if (t.is_cuda and t.dtype is dtype and t.is_contiguous()
            and t.get_device() == _device()):
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on {t.device}; the current device is "
                     f"cuda:{torch.cuda.current_device()}")


def _buffer(t: torch.Tensor, dtype, numel: int, name: str):
    """A buffer the library reads or writes through a raw pointer: as _require, and at least
    `numel` elements long, so that no kernel touches memory past its end."""
    _require(t, dtype, name)
    if t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements; {numel} are needed")
    return t


def _new(shape, dtype, device, stream):
    """A result tensor whose memory belongs to the stream that writes it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


# ------------------------------------------------------------------------- quantizer

def scale_bytes(rows: int, cols: int, axis: int = ROW, layout: int = SWIZZLED) -> int:
    n = lib().mxfp8_scale_bytes(rows, cols, axis, layout)
    if n == 0 and rows * cols != 0:
        raise ValueError(f"no scale layout for rows={rows} cols={cols} axis={axis}")
    return n


def grouped_scale_bytes(total_rows: int, cols: int, num_experts: int, axis: int = ROW) -> int:
    return lib().mxfp8_grouped_scale_bytes(total_rows, cols, num_experts, axis)


def quantize(src: torch.Tensor, axis: int = ROW, layout: int = SWIZZLED, out=None, scales=None,
             stream=None, rule: int = RULE_FLOOR):
    """MXFP8-quantize a BF16 [rows, cols] CUDA tensor. Returns (E4M3 codes as uint8, E8M0
    scale bytes as uint8): codes [rows, cols] (ROW) or [cols, rows] (COL); scales flat
    (SWIZZLED) or [S_rows, S_cols] (LINEAR)."""
    _require(src, torch.bfloat16, "src")
    rows, cols = src.shape
    oshape = (rows, cols) if axis == ROW else (cols, rows)
    if out is None:
        out = torch.empty(oshape, dtype=torch.uint8, device=src.device)
    _buffer(out, torch.uint8, rows * cols, "out")
    if scales is not None:
        _buffer(scales, torch.uint8, scale_bytes(rows, cols, axis, layout), "scales")
    else:
        nb = scale_bytes(rows, cols, axis, layout)
        if layout == LINEAR:
            s_rows, s_cols = (rows, cols // 32) if axis == ROW else (cols, rows // 32)
            scales = torch.empty((s_rows, s_cols), dtype=torch.uint8, device=src.device)
        else:
            scales = torch.empty(nb, dtype=torch.uint8, device=src.device)
    if rule == RULE_FLOOR:
        _check(lib().mxfp8_quantize(_ptr(src), rows, cols, axis, _ptr(out), _ptr(scales), layout,
                                    _stream(stream)), "mxfp8_quantize")
    else:
        _check(lib().mxfp8_quantize_rule(_ptr(src), rows, cols, axis, _ptr(out), _ptr(scales),
                                         layout, rule, _stream(stream)), "mxfp8_quantize_rule")
    return out, scales


def _alloc_scales(rows, cols, axis, layout, dev):
    if layout == LINEAR:
        s_rows, s_cols = (rows, cols // 32) if axis == ROW else (cols, rows // 32)
        return torch.empty((s_rows, s_cols), dtype=torch.uint8, device=dev)
    return torch.empty(scale_bytes(rows, cols, axis, layout), dtype=torch.uint8, device=dev)


def _dual_buffers(rows, cols, layout, row_out, row_scales, col_out, col_scales):
    _buffer(row_out, torch.uint8, rows * cols, "row_out")
    _buffer(col_out, torch.uint8, rows * cols, "col_out")
    if rows and cols:
        _buffer(row_scales, torch.uint8, scale_bytes(rows, cols, ROW, layout), "row_scales")
        _buffer(col_scales, torch.uint8, scale_bytes(rows, cols, COL, layout), "col_scales")


def quantize_dual(src: torch.Tensor, layout: int = SWIZZLED, row_out=None, row_scales=None,
                  col_out=None, col_scales=None, stream=None):
    """Row-wise and column-wise copies of a BF16 [rows, cols] tensor from one read.
    Returns (row_codes, row_scales, col_codes, col_scales)."""
    _require(src, torch.bfloat16, "src")
    rows, cols = src.shape
    dev = src.device
    row_out = torch.empty((rows, cols), dtype=torch.uint8, device=dev) if row_out is None else row_out
    col_out = torch.empty((cols, rows), dtype=torch.uint8, device=dev) if col_out is None else col_out
    if row_scales is None:
        row_scales = _alloc_scales(rows, cols, ROW, layout, dev)
    if col_scales is None:
        col_scales = _alloc_scales(rows, cols, COL, layout, dev)
    _dual_buffers(rows, cols, layout, row_out, row_scales, col_out, col_scales)
    _check(lib().mxfp8_quantize_dual(_ptr(src), rows, cols, _ptr(row_out), _ptr(row_scales),
                                     _ptr(col_out), _ptr(col_scales), layout, _stream(stream)),
           "mxfp8_quantize_dual")
    return row_out, row_scales, col_out, col_scales


BW_FP32, BW_POW2 = 0, 1  # mxfp8_blockwise_scale


def quantize_blockwise(src: torch.Tensor, scale_type: int = BW_FP32, out=None, scale_inv=None,
                       stream=None):
    """FP8 block-wise weight quantization (128 x 128 blocks). Returns (E4M3 codes as uint8
    [rows, cols], float32 scale_inv [ceil(rows/128), ceil(cols/128)])."""
    _require(src, torch.bfloat16, "src")
    rows, cols = src.shape
    dev = src.device
    out = torch.empty((rows, cols), dtype=torch.uint8, device=dev) if out is None else out
    if scale_inv is None:
        scale_inv = torch.empty(((rows + 127) // 128, (cols + 127) // 128), dtype=torch.float32,
                                device=dev)
    _buffer(out, torch.uint8, rows * cols, "out")
    _buffer(scale_inv, torch.float32, ((rows + 127) // 128) * ((cols + 127) // 128), "scale_inv")
    _check(lib().mxfp8_quantize_blockwise(_ptr(src), rows, cols, _ptr(out), _ptr(scale_inv),
                                          scale_type, _stream(stream)),
           "mxfp8_quantize_blockwise")
    return out, scale_inv


def _blockwise_1d_buffers(rows, cols, axis, dev, out, scale_inv, names, stream):
    """Codes and scales of one 1 x 128 copy: given ones checked, absent ones allocated."""
    if axis == ROW:
        oshape, sshape = (rows, cols), ((cols + 127) // 128, rows)
    else:
        oshape, sshape = (cols, (rows + 15) // 16 * 16), ((rows + 127) // 128, cols)
    if out is None:
        out = _new(oshape, torch.uint8, dev, stream)
    else:
        _buffer(out, torch.uint8, oshape[0] * oshape[1], names[0])
    if scale_inv is None:
        scale_inv = _new(sshape, torch.float32, dev, stream)
    else:
        _buffer(scale_inv, torch.float32, sshape[0] * sshape[1], names[1])
    return out, scale_inv


def quantize_blockwise_1d(src: torch.Tensor, axis: int = ROW, scale_type: int = BW_FP32,
                          out=None, scale_inv=None, stream=None):
    """FP8 block-wise quantization with 1 x 128 blocks along one axis (activations and
    gradients of blockwise_gemm). Returns (E4M3 codes as uint8, float32 scale_inv): ROW:
    [rows, cols] and [ceil(cols/128), rows]; COL (transposed): [cols, rows rounded up to 16]
    with zero codes past `rows`, and [ceil(rows/128), cols]."""
    _require(src, torch.bfloat16, "src")
    rows, cols = src.shape
    if axis not in (ROW, COL):
        raise ValueError(f"axis must be ROW or COL, got {axis}")
    out, scale_inv = _blockwise_1d_buffers(rows, cols, axis, src.device, out, scale_inv,
                                           ("out", "scale_inv"), stream)
    _check(lib().mxfp8_quantize_blockwise_1d(_ptr(src), rows, cols, axis, _ptr(out),
                                             _ptr(scale_inv), scale_type, _stream(stream)),
           "mxfp8_quantize_blockwise_1d")
    return out, scale_inv


def quantize_blockwise_1d_dual(src: torch.Tensor, scale_type: int = BW_FP32, row_out=None,
                               row_scale_inv=None, col_out=None, col_scale_inv=None,
                               stream=None):
    """quantize_blockwise_1d ROW and COL from one read. Returns (row_codes, row_scale_inv,
    col_codes, col_scale_inv)."""
    _require(src, torch.bfloat16, "src")
    rows, cols = src.shape
    row_out, row_scale_inv = _blockwise_1d_buffers(rows, cols, ROW, src.device, row_out,
                                                   row_scale_inv, ("row_out", "row_scale_inv"),
                                                   stream)
    col_out, col_scale_inv = _blockwise_1d_buffers(rows, cols, COL, src.device, col_out,
                                                   col_scale_inv, ("col_out", "col_scale_inv"),
                                                   stream)
    _check(lib().mxfp8_quantize_blockwise_1d_dual(_ptr(src), rows, cols, _ptr(row_out),
                                                  _ptr(row_scale_inv), _ptr(col_out),
                                                  _ptr(col_scale_inv), scale_type,
                                                  _stream(stream)),
           "mxfp8_quantize_blockwise_1d_dual")
    return row_out, row_scale_inv, col_out, col_scale_inv


def quantize_blockwise_dual(src: torch.Tensor, scale_type: int = BW_FP32, out=None,
                            scale_inv=None, out_t=None, scale_inv_t=None, stream=None):
    """quantize_blockwise and the transpose of its result from one read (rows and cols
    multiples of 16): a weight for the forward and the data-gradient product. Returns (codes
    [rows, cols], scale_inv, codes_t [cols, rows], scale_inv_t)."""
    _require(src, torch.bfloat16, "src")
    rows, cols = src.shape
    rb, cb, dev = (rows + 127) // 128, (cols + 127) // 128, src.device
    out = _new((rows, cols), torch.uint8, dev, stream) if out is None else out
    out_t = _new((cols, rows), torch.uint8, dev, stream) if out_t is None else out_t
    if scale_inv is None:
        scale_inv = _new((rb, cb), torch.float32, dev, stream)
    if scale_inv_t is None:
        scale_inv_t = _new((cb, rb), torch.float32, dev, stream)
    _buffer(out, torch.uint8, rows * cols, "out")
    _buffer(out_t, torch.uint8, rows * cols, "out_t")
    _buffer(scale_inv, torch.float32, rb * cb, "scale_inv")
    _buffer(scale_inv_t, torch.float32, rb * cb, "scale_inv_t")
    _check(lib().mxfp8_quantize_blockwise_dual(_ptr(src), rows, cols, _ptr(out),
                                               _ptr(scale_inv), _ptr(out_t), _ptr(scale_inv_t),
                                               scale_type, _stream(stream)),
           "mxfp8_quantize_blockwise_dual")
    return out, scale_inv, out_t, scale_inv_t


class DualJob(ctypes.Structure):
    """mxfp8_dual_job (include/mxfp8.h)."""
    _fields_ = [("src", _P), ("rows", _I64), ("cols", _I64), ("row_out", _P),
                ("row_scales", _P), ("col_out", _P), ("col_scales", _P)]


MAX_DUAL_JOBS = 8


def quantize_dual_multi(srcs, layout: int = SWIZZLED, outs=None, stream=None):
    """quantize_dual for several BF16 tensors in one launch. `outs`, if given, holds one
    (row_codes, row_scales, col_codes, col_scales) tuple per source. Returns the list of
    such tuples."""
    if not 1 <= len(srcs) <= MAX_DUAL_JOBS:
        raise ValueError(f"1 to {MAX_DUAL_JOBS} tensors per call")
    result = []
    jobs = (DualJob * len(srcs))()
    for i, src in enumerate(srcs):
        _require(src, torch.bfloat16, "src")
        rows, cols = src.shape
        dev = src.device
        if outs is not None:
            ro, rs, co, cs = outs[i]
            _dual_buffers(rows, cols, layout, ro, rs, co, cs)
        else:
            ro = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
            co = torch.empty((cols, rows), dtype=torch.uint8, device=dev)
            rs = _alloc_scales(rows, cols, ROW, layout, dev)
            cs = _alloc_scales(rows, cols, COL, layout, dev)
        jobs[i] = DualJob(src.data_ptr(), rows, cols, ro.data_ptr(), rs.data_ptr(),
                          co.data_ptr(), cs.data_ptr())
        result.append((ro, rs, co, cs))
    _check(lib().mxfp8_quantize_dual_multi(ctypes.cast(jobs, _P), len(srcs), layout,
                                           _stream(stream)), "mxfp8_quantize_dual_multi")
    return result


def quantize_grouped_dual(src: torch.Tensor, offsets: torch.Tensor, row_out=None,
                          row_scales=None, col_out=None, col_scales=None, stream=None):
    """mxfp8_quantize_grouped ROW and COL from one read. Returns
    (row_codes, row_scales, col_codes, col_scales)."""
    _require(src, torch.bfloat16, "src")
    _require(offsets, torch.int32, "offsets")
    total, cols = src.shape
    e = offsets.numel() - 1
    dev = src.device
    row_out = torch.empty((total, cols), dtype=torch.uint8, device=dev) if row_out is None else row_out
    col_out = torch.empty((cols, total), dtype=torch.uint8, device=dev) if col_out is None else col_out
    if row_scales is None:
        row_scales = torch.empty(grouped_scale_bytes(total, cols, e, ROW), dtype=torch.uint8,
                                 device=dev)
    if col_scales is None:
        col_scales = torch.empty(grouped_scale_bytes(total, cols, e, COL), dtype=torch.uint8,
                                 device=dev)
    _buffer(row_out, torch.uint8, total * cols, "row_out")
    _buffer(col_out, torch.uint8, total * cols, "col_out")
    _buffer(row_scales, torch.uint8, grouped_scale_bytes(total, cols, e, ROW), "row_scales")
    _buffer(col_scales, torch.uint8, grouped_scale_bytes(total, cols, e, COL), "col_scales")
    _check(lib().mxfp8_quantize_grouped_dual(_ptr(src), total, cols, _ptr(offsets), e,
                                             _ptr(row_out), _ptr(row_scales), _ptr(col_out),
                                             _ptr(col_scales), _stream(stream)),
           "mxfp8_quantize_grouped_dual")
    return row_out, row_scales, col_out, col_scales


def quantize_batched(src: torch.Tensor, axis: int = ROW, layout: int = SWIZZLED, out=None,
                     scales=None, stream=None):
    """Quantize each of `batch` BF16 matrices [batch, rows, cols] independently; scale
    blocks concatenated in batch order."""
    _require(src, torch.bfloat16, "src")
    batch, rows, cols = src.shape
    oshape = (batch, rows, cols) if axis == ROW else (batch, cols, rows)
    if out is None:
        out = torch.empty(oshape, dtype=torch.uint8, device=src.device)
    if scales is None:
        scales = torch.empty(batch * scale_bytes(rows, cols, axis, layout), dtype=torch.uint8,
                             device=src.device)
    _buffer(out, torch.uint8, batch * rows * cols, "out")
    if rows and cols:
        _buffer(scales, torch.uint8, batch * scale_bytes(rows, cols, axis, layout), "scales")
    _check(lib().mxfp8_quantize_batched(_ptr(src), batch, rows, cols, axis, _ptr(out),
                                        _ptr(scales), layout, _stream(stream)),
           "mxfp8_quantize_batched")
    return out, scales


def quantize_grouped(src: torch.Tensor, offsets: torch.Tensor, axis: int = ROW, out=None,
                     scales=None, stream=None):
    """Quantize a token-segmented BF16 [total_rows, cols] tensor (expert e owns rows
    offsets[e]..offsets[e+1], int32 CUDA tensor); per-expert swizzled scale blocks."""
    _require(src, torch.bfloat16, "src")
    _require(offsets, torch.int32, "offsets")
    total, cols = src.shape
    e = offsets.numel() - 1
    oshape = (total, cols) if axis == ROW else (cols, total)
    if out is None:
        out = torch.empty(oshape, dtype=torch.uint8, device=src.device)
    if scales is None:
        scales = torch.empty(grouped_scale_bytes(total, cols, e, axis), dtype=torch.uint8,
                             device=src.device)
    _buffer(out, torch.uint8, total * cols, "out")
    _buffer(scales, torch.uint8, grouped_scale_bytes(total, cols, e, axis), "scales")
    _check(lib().mxfp8_quantize_grouped(_ptr(src), total, cols, axis, _ptr(offsets), e,
                                        _ptr(out), _ptr(scales), _stream(stream)),
           "mxfp8_quantize_grouped")
    return out, scales


# ----------------------------------------------------------------------------- GEMMs

def gemm(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor, sb: torch.Tensor, op: int = FPROP,
         out_dtype: int = OUT_BF16, out=None, stream=None, workspace=None) -> torch.Tensor:
    """C[M, N] = deq(A)[M, K] . deq(B)[N, K]^T with swizzled scales (both K-major). With a
    `workspace` (a zero-filled, 32-byte aligned uint8 CUDA tensor of gemm_workspace_bytes(...)
    bytes, used by one GEMM at a time) the last wave of tiles may run as split-K pieces (mxfp8_gemm_ws)."""
    _require(a, torch.uint8, "A")
    _require(b, torch.uint8, "B")
    m, k = a.shape
    n, k2 = b.shape
    if k != k2:
        raise ValueError(f"K mismatch: {k} vs {k2}")
    dt = torch.bfloat16 if out_dtype == OUT_BF16 else torch.float32
    if out is None:
        out = torch.empty((m, n), dtype=dt, device=a.device)
    _buffer(out, dt, m * n, "out")
    if m and n and k:  # the scales are read only when there is a reduction to run
        _buffer(sa, torch.uint8, scale_bytes(m, k, ROW, SWIZZLED), "sA")
        _buffer(sb, torch.uint8, scale_bytes(n, k, ROW, SWIZZLED), "sB")
    if workspace is None:
        _check(lib().mxfp8_gemm(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(out), m, n, k, op,
                                out_dtype, _stream(stream)), "mxfp8_gemm")
    else:
        _require(workspace, torch.uint8, "workspace")
        _check(lib().mxfp8_gemm_ws(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(out), m, n, k, op,
                                   out_dtype, _ptr(workspace), workspace.numel(),
                                   _stream(stream)), "mxfp8_gemm_ws")
    return out


def gemm_workspace_bytes(m: int, n: int, k: int, op: int = FPROP, out_dtype: int = OUT_BF16) -> int:
    """Bytes of workspace with which gemm(..., workspace=...) runs the split-K last wave on
    the current device (0: it never does)."""
    return int(lib().mxfp8_gemm_workspace_bytes(m, n, k, op, out_dtype))


def grouped_gemm(a, sa, b, sb, offsets: torch.Tensor, op: int = FPROP,
                 out_dtype: int = OUT_BF16, out=None, stream=None) -> torch.Tensor:
    """Grouped expert GEMMs (see mxfp8_grouped_gemm). FPROP/DGRAD: a [T, K], b [E, N, K]
    -> [T, N]. WGRAD: a [N, T], b [K, T] -> [E, N, K]."""
    _require(a, torch.uint8, "A")
    _require(b, torch.uint8, "B")
    _require(offsets, torch.int32, "offsets")
    e = offsets.numel() - 1
    dt = torch.bfloat16 if out_dtype == OUT_BF16 else torch.float32
    if op == WGRAD:
        n_, total = a.shape
        k_ = b.shape[0]
        shape = (e, n_, k_)
    else:
        total, k_ = a.shape
        n_ = b.shape[1]
        shape = (total, n_)
    if out is None:
        out = torch.empty(shape, dtype=dt, device=a.device)
    _buffer(out, dt, shape[0] * shape[1] * (shape[2] if len(shape) == 3 else 1), "out")
    if total and n_ and k_:  # the scales are read only when there is a reduction to run
        if op == WGRAD:
            _buffer(sa, torch.uint8, grouped_scale_bytes(total, n_, e, COL), "sA")
            _buffer(sb, torch.uint8, grouped_scale_bytes(total, k_, e, COL), "sB")
        else:
            _buffer(sa, torch.uint8, grouped_scale_bytes(total, k_, e, ROW), "sA")
            _buffer(b, torch.uint8, e * n_ * k_, "B")
            _buffer(sb, torch.uint8, e * scale_bytes(n_, k_, ROW, SWIZZLED), "sB")
    _check(lib().mxfp8_grouped_gemm(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(out),
                                    _ptr(offsets), e, total, n_, k_, op, out_dtype,
                                    _stream(stream)), "mxfp8_grouped_gemm")
    return out


def blockwise_gemm_workspace_bytes(m: int, n: int, k: int, out_dtype: int = OUT_BF16) -> int:
    """Bytes of the workspace with which blockwise_gemm runs power-of-two scales on the
    block-scaled MMA (0: it never does)."""
    return int(lib().mxfp8_blockwise_gemm_workspace_bytes(m, n, k, out_dtype))


def blockwise_gemm(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor, sb: torch.Tensor,
                   op: int = FPROP, out_dtype: int = OUT_BF16, out=None, stream=None,
                   workspace=None, scale_type: Optional[int] = None) -> torch.Tensor:
    """C[M, N] = deq(A)[M, K] . deq(B)[N, K]^T of block-wise FP8 operands (both K-major). A
    and sa as quantize_blockwise_1d writes them; B and sb as quantize_blockwise does (128 x
    128 blocks), or for WGRAD as quantize_blockwise_1d does. K % 16 == 0, N % 8 == 0. Large
    products take a workspace of blockwise_gemm_workspace_bytes(...) bytes, in which scales
    are laid out for the block-scaled MMA if all are powers of two; without one given (a uint8
    CUDA tensor) it is allocated for the call. With one that is too small, an empty one for
    instance, the scales are folded in without a look at them. So they are with
    scale_type=BW_FP32, by which a caller whose scales are not powers of two saves the look (7 us
    or more of a large product); BW_POW2 is what None does: the device looks."""
    if scale_type not in (None, BW_FP32, BW_POW2):
        raise ValueError(f"scale_type must be None, BW_FP32 or BW_POW2, got {scale_type}")
    _require(a, torch.uint8, "A")
    _require(b, torch.uint8, "B")
    m, k = a.shape
    n, k2 = b.shape
    if k != k2:
        raise ValueError(f"K mismatch: {k} vs {k2}")
    dt = torch.bfloat16 if out_dtype == OUT_BF16 else torch.float32
    if out is None:
        out = _new((m, n), dt, a.device, stream)
    else:
        _buffer(out, dt, m * n, "out")
    kb = (k + 127) // 128
    if m and n and k:  # the scales are read only when there is a reduction to run
        _buffer(sa, torch.float32, kb * m, "sA")
        _buffer(sb, torch.float32, kb * (n if op == WGRAD else (n + 127) // 128), "sB")
    look = m > 128 and scale_type != BW_FP32
    need = lib().mxfp8_blockwise_gemm_workspace_bytes(m, n, k, out_dtype) if look else 0
    if workspace is not None:
        _require(workspace, torch.uint8, "workspace")
    elif need:
        workspace = _new((need,), torch.uint8, a.device, stream)
    if need:
        _check(lib().mxfp8_blockwise_gemm_ws(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(out), m,
                                             n, k, op, out_dtype, _ptr(workspace),
                                             workspace.numel(), _stream(stream)),
               "mxfp8_blockwise_gemm_ws")
    else:
        _check(lib().mxfp8_blockwise_gemm(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(out), m, n,
                                          k, op, out_dtype, _stream(stream)),
               "mxfp8_blockwise_gemm")
    return out


# --------------------------------------------------------------- token log probabilities

MAX_TOP = 32


class TokenLogprobs(NamedTuple):
    """Result of token_logprobs, one entry (or row) per row of logits."""
    logprob: torch.Tensor                # float32 [rows]
    entropy: torch.Tensor                # float32 [rows]
    stats: torch.Tensor                  # float32 [rows, 2]: max logit, log of the sum
    top_logprob: Optional[torch.Tensor]  # float32 [rows, top], or None for top = 0
    top_id: Optional[torch.Tensor]       # int64 [rows, top], or None


def _logits(t: torch.Tensor, name: str):
    """Logits as the library takes them: 2-D, BF16 or FP32, each row contiguous, on the
    current device. Returns (dtype code, rows, vocab, row pitch)."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got {t.dim()}")
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}; the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    rows, vocab = t.shape
    pitch, step = t.stride()
    if rows <= 1:
        pitch = vocab
    if vocab > 1 and step != 1 or pitch < vocab:
        raise ValueError(f"{name} must have contiguous rows that do not overlap, got strides "
                         f"{t.stride()}")
    return OUT_BF16 if t.dtype == torch.bfloat16 else OUT_FP32, rows, vocab, pitch


def token_logprobs(logits: torch.Tensor, targets: torch.Tensor, temperature: float = 1.0,
                   top: int = 0, stream=None) -> TokenLogprobs:
    """Log probability of each row's target token under softmax(logits / temperature), the
    entropy, and the `top` (at most MAX_TOP) likeliest tokens, equal logits lowest token
    first. logits: BF16 or FP32 [rows, vocab], rows of any pitch; targets: int64 [rows],
    negative where a row is not scored (logprob 0). Masked logits are -inf; see
    include/mxfp8.h for rows with nothing left, and for NaN."""
    dt, rows, vocab, pitch = _logits(logits, "logits")
    _buffer(targets, torch.int64, rows, "targets")
    if not 0 <= top <= MAX_TOP:
        raise ValueError(f"top must be 0 to {MAX_TOP}, got {top}")
    dev = logits.device
    logprob = _new((rows,), torch.float32, dev, stream)
    entropy = _new((rows,), torch.float32, dev, stream)
    stats = _new((rows, 2), torch.float32, dev, stream)
    top_logprob = top_id = None
    if top:
        top_logprob = _new((rows, top), torch.float32, dev, stream)
        top_id = _new((rows, top), torch.int64, dev, stream)
    _check(lib().mxfp8_token_logprobs(_ptr(logits), dt, rows, vocab, pitch, _ptr(targets),
                                      temperature, _ptr(logprob), _ptr(entropy), _ptr(stats),
                                      top, _ptr(top_logprob) if top else None,
                                      _ptr(top_id) if top else None, _stream(stream)),
           "mxfp8_token_logprobs")
    return TokenLogprobs(logprob, entropy, stats, top_logprob, top_id)


def token_logprobs_backward(logits: torch.Tensor, targets: torch.Tensor, stats: torch.Tensor,
                            entropy: torch.Tensor, grad_logprob: torch.Tensor,
                            grad_entropy=None, top_id=None, grad_top=None,
                            temperature: float = 1.0, out=None, stream=None) -> torch.Tensor:
    """Gradient with respect to the logits of a loss whose gradients with respect to
    token_logprobs' logprob, entropy and top_logprob are given (float32; the last two
    optional). `stats`, `entropy` and `top_id` are that call's, `temperature` its
    temperature. The result has the logits' type, shape and row pitch; `out` may be any such
    tensor of contiguous rows, the logits themselves included (another place within 16 bytes
    than the logits' makes the call 2 to 3 times slower)."""
    dt, rows, vocab, pitch = _logits(logits, "logits")
    _buffer(targets, torch.int64, rows, "targets")
    _buffer(stats, torch.float32, 2 * rows, "stats")
    _buffer(entropy, torch.float32, rows, "entropy")
    _buffer(grad_logprob, torch.float32, rows, "grad_logprob")
    if grad_entropy is not None:
        _buffer(grad_entropy, torch.float32, rows, "grad_entropy")
    top = 0
    if (grad_top is None) != (top_id is None):
        raise ValueError("top_id and grad_top go together")
    if grad_top is not None:
        if grad_top.dim() != 2 or not 1 <= grad_top.shape[1] <= MAX_TOP:
            raise ValueError(f"grad_top must be [rows, 1 to {MAX_TOP}], got "
                             f"{tuple(grad_top.shape)}")
        top = grad_top.shape[1]
        if tuple(top_id.shape) != tuple(grad_top.shape):
            raise ValueError(f"top_id is {tuple(top_id.shape)}; grad_top is "
                             f"{tuple(grad_top.shape)}")
        _buffer(grad_top, torch.float32, rows * top, "grad_top")
        _buffer(top_id, torch.int64, rows * top, "top_id")
    if out is None:
        out_pitch = pitch
        if stream is None:
            out = torch.empty_strided((rows, vocab), (pitch, 1), dtype=logits.dtype,
                                      device=logits.device)
        else:
            with torch.cuda.stream(stream):
                out = torch.empty_strided((rows, vocab), (pitch, 1), dtype=logits.dtype,
                                          device=logits.device)
    else:
        odt, orows, ovocab, out_pitch = _logits(out, "out")
        if (odt, orows, ovocab) != (dt, rows, vocab):
            raise ValueError(f"out must be {logits.dtype} {tuple(logits.shape)}, got {out.dtype} "
                             f"{tuple(out.shape)}")
    _check(lib().mxfp8_token_logprobs_backward(
        _ptr(logits), dt, rows, vocab, pitch, _ptr(targets), temperature, _ptr(stats),
        _ptr(entropy), _ptr(grad_logprob), None if grad_entropy is None else _ptr(grad_entropy),
        top, _ptr(top_id) if top else None, _ptr(grad_top) if top else None, _ptr(out),
        out_pitch, _stream(stream)), "mxfp8_token_logprobs_backward")
    return out


# ------------------------------------------------------------- routing tokens to experts

_INT32, _FP32, _BF16 = torch.int32, torch.float32, torch.bfloat16


class RoutePlan(NamedTuple):
    """Entries (token, choice) sorted by expert into segments padded to 32 rows (route). All
    int32, on the device."""
    offsets: torch.Tensor   # [num_experts + 1], as quantize_grouped and grouped_gemm take them
    row_of: torch.Tensor    # [tokens, top_k], the row of each entry; -1: of no expert
    entry_of: torch.Tensor  # [rows], the entry (token * top_k + choice) of each row; -1: padding


_MOST_ROUTED, _MOST_EXPERTS = 0x7FFFFF00, 1024   # mxfp8_route's limits


def route_rows(tokens: int, top_k: int, num_experts: int) -> int:
    """Rows that the segments of any choice of experts fit in."""
    rows = 0
    if 0 < tokens <= _MOST_ROUTED >= top_k > 0 < num_experts <= _MOST_EXPERTS:   # C's types hold them
        rows = int(lib().mxfp8_route_rows(tokens, top_k, num_experts))
    if rows == 0 and tokens != 0:
        raise ValueError(f"no segments for tokens={tokens} top_k={top_k} "
                         f"num_experts={num_experts}")
    return rows


def _plan_rows(n, experts):
    """mxfp8_route_rows of n entries, fewer than 2^30, without the call."""
    return (n + 31 * min(n, experts)) // 32 * 32


def route(ids: torch.Tensor, num_experts: int, rows: Optional[int] = None,
          stream=None) -> RoutePlan:
    """Sorts the entries of ids (int64 [tokens, top_k], negative: of no expert) by expert, each
    expert's in their order. `rows` (default: route_rows, which any choice fits) may be fewer
    where the caller knows the experts' counts; the last segment takes what is left over."""
    _require(ids, torch.int64, "ids")
    if ids.dim() != 2 or ids.shape[1] < 1:
        raise ValueError(f"ids must be [tokens, top_k], got {tuple(ids.shape)}")
    tokens, top_k = ids.shape
    if top_k > _MOST_ROUTED or not 0 < num_experts <= _MOST_EXPERTS:
        if rows is None:
            route_rows(tokens, top_k, num_experts)
        _check(ERR_INVALID_ARG, "mxfp8_route")
    n = tokens * top_k
    if rows is None:
        if n < 1 << 30:
            rows = _plan_rows(n, num_experts)
        else:
            rows = route_rows(tokens, top_k, num_experts)
    elif rows < 0:
        raise ValueError(f"rows must not be negative, got {rows}")
    dev = ids.device
    offsets = _new((num_experts + 1,), torch.int32, dev, stream)
    row_of = _new((tokens, top_k), torch.int32, dev, stream)
    entry_of = _new((rows,), torch.int32, dev, stream)
    _check(lib().mxfp8_route(_ptr(ids), tokens, top_k, num_experts, rows, _ptr(offsets),
                             _ptr(row_of), _ptr(entry_of), _here(stream)), "mxfp8_route")
    return RoutePlan(offsets, row_of, entry_of)


def _here(stream):
    """_stream, once a CUDA tensor on the current device has been seen."""
    return _raw_stream(_device()) if stream is None else stream.cuda_stream


def _plan_refused(t, plan: RoutePlan, weights, name: str):
    """Says what is wrong with a call on a plan."""
    if t.dtype not in (_BF16, _FP32):
        raise ValueError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    _require(t, t.dtype, name)
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got {t.dim()}")
    _require(plan.row_of, _INT32, "plan.row_of")
    _require(plan.entry_of, _INT32, "plan.entry_of")
    if plan.row_of.dim() != 2 or not 0 < plan.row_of.shape[1] <= _MOST_ROUTED:
        raise ValueError(f"plan.row_of must be [tokens, top_k], top_k 1 to {_MOST_ROUTED}, got "
                         f"{tuple(plan.row_of.shape)}")
    _require(weights, _FP32, "weights")
    raise ValueError(f"weights are {tuple(weights.shape)}; the plan is of "
                     f"{tuple(plan.row_of.shape)}")


def _planned(t, plan: RoutePlan, weights, name: str):
    """Rows `t` of tokens or of segments, the plan and the weights beside it, checked: what is right
    passes in two expressions, as a call of a few tokens takes longer in here than on the GPU.
    Returns (tokens, top_k, rows, t's rows, its columns, its dtype)."""
    row_of, entry_of = plan.row_of, plan.entry_of
    dt, dev, of = t.dtype, t.get_device(), row_of.shape
    if not ((dt is _BF16 or dt is _FP32) and row_of.dtype is _INT32 is entry_of.dtype
            and dev >= 0 and dev == _device() == row_of.get_device() == entry_of.get_device()
            and t.is_contiguous() and row_of.is_contiguous() and entry_of.is_contiguous()
            and len(of) == 2 and 0 < of[1] <= _MOST_ROUTED and t.dim() == 2) or (
            weights is not None and not (
                weights.dtype is _FP32 and weights.get_device() == dev
                and weights.is_contiguous() and weights.shape == of)):
        _plan_refused(t, plan, weights, name)
    return *of, entry_of.numel(), *t.shape, dt


def _optional(t):
    return None if t is None else t.data_ptr()


def dispatch(x: torch.Tensor, plan: RoutePlan, weights: Optional[torch.Tensor] = None, out=None,
             stream=None) -> torch.Tensor:
    """The tokens' rows x (BF16 or FP32 [tokens, cols]) in the plan's segments, [rows, cols]: row
    r holds its entry's token, times that entry's weight (float32 [tokens, top_k]) if given;
    padding rows are zero. The gradient of x without weights is combine(grad, plan)."""
    tokens, top_k, rows, n, cols, dt = _planned(x, plan, weights, "x")
    if n != tokens:
        raise ValueError(f"x has {n} rows; the plan is of {tokens} tokens")
    if out is None:
        out = _new((rows, cols), dt, x.device, stream)
    else:
        _buffer(out, dt, rows * cols, "out")
    _check(lib().mxfp8_dispatch(x.data_ptr(), OUT_BF16 if dt is _BF16 else OUT_FP32, tokens, cols,
                                top_k, _optional(weights), plan.row_of.data_ptr(),
                                plan.entry_of.data_ptr(), rows, out.data_ptr(), _here(stream)),
           "mxfp8_dispatch")
    return out


def _copy_scale_bytes(rows, cols, experts, axis):
    """mxfp8_grouped_scale_bytes, without the call for the usual sizes."""
    if experts > 0 and rows % 32 == 0 == cols % 32:
        return (-(-rows // 128) + experts) * -(-cols // 128) * 512
    return lib().mxfp8_grouped_scale_bytes(rows, cols, experts, axis)


def _dispatch_copy(rows, cols, experts, axis, codes, scales, device, stream):
    """Codes and scales of one grouped copy: given ones checked, absent ones allocated."""
    need = _copy_scale_bytes(rows, cols, experts, axis)
    if need == 0 and cols:   # cols not a multiple of 32, or sizes that do not fit: as the call says
        _check(ERR_ALIGNMENT if axis == ROW and cols % 32 else ERR_INVALID_ARG,
               "mxfp8_quantize_dispatch")
    if codes is None:
        codes = _new((rows, cols) if axis == ROW else (cols, rows), torch.uint8, device, stream)
    else:
        _buffer(codes, torch.uint8, rows * cols, "codes")
    if scales is None:
        scales = _new((need,), torch.uint8, device, stream)
    else:
        _buffer(scales, torch.uint8, need, "scales")
    return codes, scales


def _dispatch_source(x, plan, weights):
    """Checks quantize_dispatch's inputs. Returns (tokens, top_k, rows, cols, experts)."""
    tokens, top_k, rows, n, cols, dt = _planned(x, plan, weights, "x")
    if n != tokens:
        raise ValueError(f"x has {n} rows; the plan is of {tokens} tokens")
    if dt is not _BF16:
        raise ValueError(f"x must be torch.bfloat16, got {dt}")
    offsets = plan.offsets
    _require(offsets, _INT32, "plan.offsets")
    return tokens, top_k, rows, cols, offsets.numel() - 1


def quantize_dispatch(x: torch.Tensor, plan: RoutePlan, axis: int = ROW,
                      weights: Optional[torch.Tensor] = None, out=None, scales=None, stream=None):
    """quantize_grouped(dispatch(x, plan, weights), plan.offsets, axis) in one pass, byte for
    byte (x BF16 [tokens, cols]). Returns (codes, scales); scale bytes past the last segment's
    are zero."""
    if axis not in (ROW, COL):
        raise ValueError(f"axis must be ROW or COL, got {axis}")
    tokens, top_k, rows, cols, e = _dispatch_source(x, plan, weights)
    codes, scales = _dispatch_copy(rows, cols, e, axis, out, scales, x.device, stream)
    a, b = codes.data_ptr(), scales.data_ptr()
    ra, rb, ca, cb = (a, b, None, None) if axis == ROW else (None, None, a, b)
    _check(lib().mxfp8_quantize_dispatch(x.data_ptr(), tokens, cols, top_k, _optional(weights),
                                         plan.row_of.data_ptr(), plan.entry_of.data_ptr(), rows,
                                         plan.offsets.data_ptr(), e, ra, rb, ca, cb,
                                         _here(stream)), "mxfp8_quantize_dispatch")
    return codes, scales


def quantize_dispatch_dual(x: torch.Tensor, plan: RoutePlan,
                           weights: Optional[torch.Tensor] = None, row_out=None, row_scales=None,
                           col_out=None, col_scales=None, stream=None):
    """quantize_dispatch ROW and COL in one call. Returns (row_codes, row_scales, col_codes,
    col_scales): an expert layer's forward and weight-gradient operands; with x the gradient of
    combine's result and its weights, the operands of the layer before it."""
    tokens, top_k, rows, cols, e = _dispatch_source(x, plan, weights)
    row = _dispatch_copy(rows, cols, e, ROW, row_out, row_scales, x.device, stream)
    col = _dispatch_copy(rows, cols, e, COL, col_out, col_scales, x.device, stream)
    _check(lib().mxfp8_quantize_dispatch(x.data_ptr(), tokens, cols, top_k, _optional(weights),
                                         plan.row_of.data_ptr(), plan.entry_of.data_ptr(), rows,
                                         plan.offsets.data_ptr(), e, row[0].data_ptr(),
                                         row[1].data_ptr(), col[0].data_ptr(), col[1].data_ptr(),
                                         _here(stream)), "mxfp8_quantize_dispatch")
    return row + col


def combine(y: torch.Tensor, plan: RoutePlan, weights: Optional[torch.Tensor] = None, out=None,
            stream=None) -> torch.Tensor:
    """The sum of each token's segment rows y (BF16 or FP32 [rows, cols]), weighted (float32
    [tokens, top_k]) if weights are given, [tokens, cols] of y's type: FP32 sums in the order of
    the choices, rounded once. A token without rows gets zeros."""
    tokens, top_k, rows, n, cols, dt = _planned(y, plan, weights, "y")
    if n != rows:
        raise ValueError(f"y has {n} rows; the plan has {rows}")
    if out is None:
        out = _new((tokens, cols), dt, y.device, stream)
    else:
        _buffer(out, dt, tokens * cols, "out")
    _check(lib().mxfp8_combine(y.data_ptr(), OUT_BF16 if dt is _BF16 else OUT_FP32, rows, cols,
                               tokens, top_k, _optional(weights), plan.row_of.data_ptr(),
                               out.data_ptr(), _here(stream)), "mxfp8_combine")
    return out


def combine_backward(grad_out: torch.Tensor, y: torch.Tensor, plan: RoutePlan,
                     weights: torch.Tensor, grad_rows: bool = True, out=None, out_weights=None,
                     stream=None):
    """Gradients of combine(y, plan, weights): (grad_y [rows, cols] of y's type, padding rows
    zero; grad_weights float32 [tokens, top_k]). grad_rows=False leaves the first out (None):
    quantize_dispatch_dual(grad_out, plan, weights) gives it as the grouped GEMMs read it."""
    if weights is None:
        raise ValueError("weights are needed; without them grad_y is dispatch(grad_out, plan)")
    tokens, top_k, rows, n, cols, dt = _planned(y, plan, weights, "y")
    if n != rows:
        raise ValueError(f"y has {n} rows; the plan has {rows}")
    _require(grad_out, dt, "grad_out")
    if grad_out.shape != (tokens, cols):
        raise ValueError(f"grad_out must be {(tokens, cols)}, got {tuple(grad_out.shape)}")
    if not grad_rows:
        if out is not None:
            raise ValueError("out is given, but grad_rows is False")
    elif out is None:
        out = _new((rows, cols), dt, y.device, stream)
    else:
        _buffer(out, dt, rows * cols, "out")
    if out_weights is None:
        out_weights = _new((tokens, top_k), torch.float32, y.device, stream)
    else:
        _buffer(out_weights, torch.float32, tokens * top_k, "out_weights")
    _check(lib().mxfp8_combine_backward(grad_out.data_ptr(), y.data_ptr(),
                                        OUT_BF16 if dt is _BF16 else OUT_FP32, tokens, cols,
                                        top_k, weights.data_ptr(), plan.row_of.data_ptr(),
                                        plan.entry_of.data_ptr(), rows, _optional(out),
                                        out_weights.data_ptr(), _here(stream)),
           "mxfp8_combine_backward")
    return out, out_weights


# ------------------------------------------------------- gated activation, 8-bit checkpoint

class Swiglu(NamedTuple):
    """Result of swiglu."""
    h: torch.Tensor                 # BF16 [rows, width]
    codes: Optional[torch.Tensor]   # E4M3 as uint8 [rows, 2 * width], or None
    scales: Optional[torch.Tensor]  # E8M0 bytes [rows, 2 * width / 32], or None


def swiglu(gate_up: torch.Tensor, checkpoint: bool = True, rule: int = RULE_CEIL, out=None,
           codes=None, scales=None, stream=None) -> Swiglu:
    """h = silu(gate) * up of a BF16 [rows, 2 * width] tensor [gate | up] (width % 32 == 0), with
    gate_up kept in MXFP8 for swiglu_backward: quantize(gate_up, ROW, LINEAR, rule=rule) byte for
    byte, from the same read. checkpoint=False keeps nothing."""
    _require(gate_up, torch.bfloat16, "gate_up")
    shape = gate_up.shape
    if len(shape) != 2 or shape[1] % 64:
        raise ValueError(f"gate_up must be [rows, 2 * width], width a multiple of 32, got "
                         f"{tuple(gate_up.shape)}")
    rows, width, dev = shape[0], shape[1] // 2, gate_up.device
    if out is None:
        out = _new((rows, width), torch.bfloat16, dev, stream)
    else:
        _buffer(out, torch.bfloat16, rows * width, "out")
    if checkpoint:
        n, blocks = 2 * rows * width, width // 16
        if codes is None:
            codes = _new((rows, 2 * width), torch.uint8, dev, stream)
        else:
            _buffer(codes, torch.uint8, n, "codes")
        if scales is None:
            scales = _new((rows, blocks), torch.uint8, dev, stream)
        else:
            _buffer(scales, torch.uint8, rows * blocks, "scales")
    elif codes is not None or scales is not None:
        raise ValueError("codes or scales are given, but checkpoint is False")
    if rows and width:
        if rule not in (RULE_FLOOR, RULE_CEIL):
            _check(ERR_INVALID_ARG, "mxfp8_swiglu")
        _check(lib().mxfp8_swiglu(_ptr(gate_up), rows, width, _ptr(out), _optional(codes),
                                  _optional(scales), rule, _here(stream)), "mxfp8_swiglu")
    return Swiglu(out, codes, scales)


def swiglu_backward(grad_h: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                    recompute: bool = False, out=None, out_h=None, stream=None):
    """Gradient of swiglu with respect to gate_up, from the gradient of h (BF16 [rows, width])
    and what swiglu kept. Returns (BF16 [rows, 2 * width], h or None): with recompute=True h of
    the kept values comes too, BF16 [rows, width], for the next layer's weight gradient (out_h
    may be grad_h itself)."""
    _require(grad_h, torch.bfloat16, "grad_h")
    if grad_h.dim() != 2 or grad_h.shape[1] % 32:
        raise ValueError(f"grad_h must be [rows, width], width a multiple of 32, got "
                         f"{tuple(grad_h.shape)}")
    rows, width = grad_h.shape
    _buffer(codes, torch.uint8, 2 * rows * width, "codes")
    _buffer(scales, torch.uint8, rows * (width // 16), "scales")
    if out is None:
        out = _new((rows, 2 * width), torch.bfloat16, grad_h.device, stream)
    else:
        _buffer(out, torch.bfloat16, 2 * rows * width, "out")
    if not recompute:
        if out_h is not None:
            raise ValueError("out_h is given, but recompute is False")
    elif out_h is None:
        out_h = _new((rows, width), torch.bfloat16, grad_h.device, stream)
    else:
        _buffer(out_h, torch.bfloat16, rows * width, "out_h")
    _check(lib().mxfp8_swiglu_backward(_ptr(grad_h), _ptr(codes), _ptr(scales), rows, width,
                                       _ptr(out), _optional(out_h), _here(stream)),
           "mxfp8_swiglu_backward")
    return out, out_h


SELF_CHECK_TOLERANCE = 0.25  # section "Correctness: how it fails": the self-check's tolerance


def selfcheck(w_codes: torch.Tensor, w_scales: torch.Tensor, ref_codes: torch.Tensor,
              ref_scales: torch.Tensor, x: torch.Tensor, workspace=None,
              stream=None) -> torch.Tensor:
    """Relative error ||Y - Y_ref|| / ||Y_ref|| of the MXFP8 layer as the GEMM reads it
    (w_codes + swizzled w_scales) on the quantized input x, against x times the canonical
    synchronized weight (ref_codes + linear ref_scales) dequantized. Returns a one-element
    float32 CUDA tensor (no host synchronization); compare with SELF_CHECK_TOLERANCE."""
    _require(w_codes, torch.uint8, "w_codes")
    _require(ref_codes, torch.uint8, "ref_codes")
    _require(x, torch.bfloat16, "x")
    n, k = w_codes.shape
    t = x.shape[0]
    need = lib().mxfp8_selfcheck_workspace_bytes(t, n, k)
    if need == 0:
        raise ValueError(f"no self-check for tokens={t} N={n} K={k}")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    _buffer(w_scales, torch.uint8, scale_bytes(n, k, ROW, SWIZZLED), "w_scales")
    _buffer(ref_codes, torch.uint8, n * k, "ref_codes")
    _buffer(ref_scales, torch.uint8, n * (k // 32), "ref_scales")
    _buffer(workspace, torch.uint8, need, "workspace")
    if x.shape[1] != k:
        raise ValueError(f"x has {x.shape[1]} columns; the weight has K = {k}")
    out = torch.empty(1, dtype=torch.float32, device=x.device)
    _check(lib().mxfp8_selfcheck(_ptr(w_codes), _ptr(w_scales), _ptr(ref_codes),
                                 _ptr(ref_scales), n, k, _ptr(x), t, _ptr(workspace),
                                 workspace.numel(), _ptr(out), _stream(stream)),
           "mxfp8_selfcheck")
    return out


def set_wait_limit_ns(ns: int = 0) -> None:
    """Pipeline wait limit of later GEMM launches, in nanoseconds (0: the default, 4 s or
    MXFP8_WAIT_LIMIT_MS); a kernel whose wait runs out latches ERR_TIMEOUT."""
    _check(lib().mxfp8_set_wait_limit_ns(ns), "mxfp8_set_wait_limit_ns")


def device_status(stream=None) -> int:
    """Synchronizes the stream and returns-and-clears the device status word."""
    return lib().mxfp8_get_device_status(_stream(stream))
