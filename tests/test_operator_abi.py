"""Host-side refusals of the block-wise GEMM, its quantizers and the token log probabilities:
every call here fails a check, or is empty, before anything touches a device."""
import ctypes

import pytest

import __graft_entry__
import mxfp8_block_scaled_05_gb300 as m

P = ctypes.c_void_p(0x10000)          # never dereferenced
ODD = ctypes.c_void_p(0x10001)
HALF = ctypes.c_void_p(0x10008)
BIG = 2 ** 62


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return m.lib()


def test_status_text(lib):
    assert b"target" in lib.mxfp8_status_string(m.ERR_BAD_TARGET)


def test_quantize_blockwise_1d(lib):
    q = lib.mxfp8_quantize_blockwise_1d
    assert q(P, 5, 24, m.ROW, P, P, 0, None) == m.ERR_ALIGNMENT       # cols % 16
    assert q(P, 5, 12, m.COL, P, P, 0, None) == m.ERR_ALIGNMENT       # cols % 8
    assert q(P, 5, 32, 2, P, P, 0, None) == m.ERR_INVALID_ARG
    assert q(P, 5, 32, m.ROW, P, P, 2, None) == m.ERR_INVALID_ARG
    assert q(P, -1, 32, m.ROW, P, P, 0, None) == m.ERR_INVALID_ARG
    assert q(None, 5, 32, m.ROW, P, P, 0, None) == m.ERR_INVALID_ARG
    assert q(P, 5, 32, m.ROW, None, P, 0, None) == m.ERR_INVALID_ARG
    assert q(P, 5, 32, m.COL, P, None, 0, None) == m.ERR_INVALID_ARG
    assert q(HALF, 5, 32, m.ROW, P, P, 0, None) == m.ERR_ALIGNMENT
    assert q(P, 5, 32, m.ROW, HALF, P, 0, None) == m.ERR_ALIGNMENT
    assert q(P, 5, 32, m.ROW, P, ODD, 0, None) == m.ERR_ALIGNMENT
    assert q(P, 65536 * 128, 32, m.ROW, P, P, 0, None) == m.ERR_INVALID_ARG
    assert q(P, 5, BIG, m.ROW, P, P, 0, None) == m.ERR_INVALID_ARG
    assert q(None, 0, 32, m.ROW, None, None, 0, None) == m.OK
    assert q(None, 5, 0, m.COL, None, None, 0, None) == m.OK


def test_dual_quantizers(lib):
    for q in (lib.mxfp8_quantize_blockwise_1d_dual, lib.mxfp8_quantize_blockwise_dual):
        assert q(P, 32, 24, P, P, P, P, 0, None) == m.ERR_ALIGNMENT
        assert q(P, 32, 32, P, P, P, P, 9, None) == m.ERR_INVALID_ARG
        assert q(P, 32, 32, P, P, None, P, 0, None) == m.ERR_INVALID_ARG
        assert q(P, 32, 32, P, P, P, None, 0, None) == m.ERR_INVALID_ARG
        assert q(P, 32, 32, P, P, HALF, P, 0, None) == m.ERR_ALIGNMENT
        assert q(P, 32, 32, P, P, P, ODD, 0, None) == m.ERR_ALIGNMENT
        assert q(None, 0, 32, None, None, None, None, 0, None) == m.OK
    assert lib.mxfp8_quantize_blockwise_dual(P, 24, 32, P, P, P, P, 0, None) == m.ERR_ALIGNMENT


def test_blockwise_gemm(lib):
    g = lib.mxfp8_blockwise_gemm
    assert g(P, P, P, P, P, 4, 64, 24, 0, 0, None) == m.ERR_ALIGNMENT     # K % 16
    assert g(P, P, P, P, P, 4, 60, 32, 0, 0, None) == m.ERR_ALIGNMENT     # N % 8
    assert g(P, P, P, P, P, -4, 64, 32, 0, 0, None) == m.ERR_INVALID_ARG
    assert g(P, P, P, P, P, 4, 64, 32, 3, 0, None) == m.ERR_INVALID_ARG
    assert g(P, P, P, P, P, 4, 64, 32, 0, 2, None) == m.ERR_INVALID_ARG
    assert g(P, P, P, P, P, 2 ** 31, 64, 32, 0, 0, None) == m.ERR_INVALID_ARG
    for i in range(5):
        args = [P] * 5
        args[i] = None
        assert g(*args, 4, 64, 32, 0, 0, None) == m.ERR_INVALID_ARG
        args[i] = ODD
        assert g(*args, 4, 64, 32, 0, 0, None) == m.ERR_ALIGNMENT
    assert g(None, None, None, None, None, 0, 64, 32, 0, 0, None) == m.OK
    assert g(None, None, None, None, None, 4, 0, 32, 2, 1, None) == m.OK
    assert g(None, None, None, None, None, 4, 64, 0, 0, 0, None) == m.ERR_INVALID_ARG


def test_token_logprobs(lib):
    f = lib.mxfp8_token_logprobs

    def call(logits=P, dt=0, rows=4, vocab=100, ld=100, targets=P, t=1.0, lp=P, ent=P, stats=P,
             top=0, tl=None, ti=None):
        return f(logits, dt, rows, vocab, ld, targets, t, lp, ent, stats, top, tl, ti, None)

    bad = [dict(dt=2), dict(rows=-1), dict(vocab=0), dict(vocab=2 ** 31, ld=2 ** 31),
           dict(ld=99), dict(rows=BIG, ld=BIG), dict(top=-1), dict(top=33, tl=P, ti=P),
           dict(top=4), dict(top=4, tl=P), dict(logits=None), dict(targets=None), dict(lp=None),
           dict(ent=None), dict(stats=None), dict(t=0.0), dict(t=-1.0), dict(t=float("nan")),
           dict(t=float("inf")), dict(t=1e-300), dict(t=1e300)]
    for kw in bad:
        assert call(**kw) == m.ERR_INVALID_ARG, kw
    for kw in (dict(logits=ODD), dict(dt=1, logits=ctypes.c_void_p(0x10002)),
               dict(targets=ctypes.c_void_p(0x10004)), dict(lp=ODD), dict(ent=ODD),
               dict(stats=ODD), dict(top=2, tl=ODD, ti=P),
               dict(top=2, tl=P, ti=ctypes.c_void_p(0x10004))):
        assert call(**kw) == m.ERR_ALIGNMENT, kw
    assert call(rows=0, logits=None, targets=None, lp=None, ent=None, stats=None) == m.OK


def test_token_logprobs_backward(lib):
    f = lib.mxfp8_token_logprobs_backward

    def call(logits=P, dt=0, rows=4, vocab=100, ld=100, targets=P, t=1.0, stats=P, ent=P, gl=P,
             ge=None, top=0, ti=None, gt=None, out=ctypes.c_void_p(0x90000), out_ld=100):
        return f(logits, dt, rows, vocab, ld, targets, t, stats, ent, gl, ge, top, ti, gt, out,
                 out_ld, None)

    for kw in (dict(dt=5), dict(rows=-2), dict(ld=4), dict(out_ld=99), dict(out=None),
               dict(stats=None), dict(ent=None), dict(gl=None), dict(top=3), dict(top=3, ti=P),
               dict(top=40, ti=P, gt=P), dict(t=0.0), dict(out=P, out_ld=101),
               dict(out_ld=BIG)):
        assert call(**kw) == m.ERR_INVALID_ARG, kw
    for kw in (dict(out=ODD), dict(logits=ODD), dict(ge=ODD), dict(gl=ODD), dict(stats=ODD),
               dict(top=2, ti=ODD, gt=P), dict(top=2, ti=P, gt=ODD)):
        assert call(**kw) == m.ERR_ALIGNMENT, kw
    assert call(rows=0, out=None) == m.OK
