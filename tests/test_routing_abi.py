"""Host-side refusals of the routing calls and of the gated activation, from C and from Python:
every call here fails a check, or is empty, before anything touches a device."""
import ctypes

import pytest
import torch

import __graft_entry__
import mxfp8_block_scaled_05_gb300 as m
import oracle.routing_oracle as R

P = ctypes.c_void_p(0x10000)          # never dereferenced
ODD = ctypes.c_void_p(0x10002)
HALF = ctypes.c_void_p(0x10008)
BIG = 2 ** 62


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return m.lib()


def test_status_text(lib):
    assert b"expert" in lib.mxfp8_status_string(m.ERR_BAD_EXPERT)


def test_route_rows(lib):
    f = lib.mxfp8_route_rows
    for t, k, e in [(1, 8, 128), (8192, 8, 128), (37, 3, 5), (1, 1, 1), (7, 2, 1024), (0, 4, 9)]:
        assert f(t, k, e) == R.rows_for(t, k, e)
    for bad in [(-1, 8, 8), (4, 0, 8), (4, 2, 0), (4, 2, 1025), (BIG, 8, 8), (2 ** 31, 1, 8),
                (0x7FFFFF00, 1, 1024)]:
        assert f(*bad) == 0
    assert m.route_rows(0, 2, 4) == 0
    with pytest.raises(ValueError, match="num_experts"):
        m.route_rows(4, 2, 0)


def test_route(lib):
    def call(ids=P, tokens=4, k=2, experts=8, rows=256, offsets=P, row_of=P, entry_of=P):
        return lib.mxfp8_route(ids, tokens, k, experts, rows, offsets, row_of, entry_of, None)

    for kw in (dict(tokens=-1), dict(k=0), dict(experts=0), dict(experts=1025), dict(rows=-32),
               dict(rows=2 ** 31), dict(tokens=BIG), dict(tokens=2 ** 31), dict(ids=None),
               dict(offsets=None), dict(row_of=None), dict(entry_of=None)):
        assert call(**kw) == m.ERR_INVALID_ARG, kw
    for kw in (dict(rows=33), dict(ids=ctypes.c_void_p(0x10004)), dict(offsets=ODD),
               dict(row_of=ODD), dict(entry_of=ODD)):
        assert call(**kw) == m.ERR_ALIGNMENT, kw


def test_dispatch(lib):
    def call(x=P, dt=0, tokens=4, cols=64, k=2, w=P, row_of=P, entry_of=P, rows=64, out=P):
        return lib.mxfp8_dispatch(x, dt, tokens, cols, k, w, row_of, entry_of, rows, out, None)

    for kw in (dict(x=None), dict(dt=2), dict(tokens=-1), dict(cols=-1), dict(cols=2 ** 31),
               dict(k=0), dict(row_of=None), dict(entry_of=None), dict(rows=-32),
               dict(rows=2 ** 31), dict(out=None), dict(tokens=BIG)):
        assert call(**kw) == m.ERR_INVALID_ARG, kw
    for kw in (dict(x=HALF), dict(w=ODD), dict(row_of=ODD), dict(entry_of=ODD), dict(rows=40),
               dict(out=HALF)):
        assert call(**kw) == m.ERR_ALIGNMENT, kw
    assert call(cols=65535 * 32 + 1) == m.ERR_INVALID_ARG
    assert call(rows=0, out=None, entry_of=None) == m.OK
    assert call(cols=0, x=None, out=None) == m.OK


def test_quantize_dispatch(lib):
    def call(x=P, tokens=4, cols=64, k=2, w=P, row_of=P, entry_of=P, rows=64, offsets=P,
             experts=4, rc=P, rs=P, cc=P, cs=P):
        return lib.mxfp8_quantize_dispatch(x, tokens, cols, k, w, row_of, entry_of, rows, offsets,
                                           experts, rc, rs, cc, cs, None)

    none = dict(rc=None, rs=None)
    for kw in (dict(x=None), dict(tokens=-1), dict(k=0), dict(row_of=None),
               dict(entry_of=None), dict(rows=-32), dict(offsets=None), dict(experts=0), dict(experts=1025), dict(rc=None),
               dict(rs=None), dict(cc=None), dict(cs=None), dict(cols=-32),
               dict(rc=None, rs=None, cc=None, cs=None), dict(rows=65535 * 128),
               dict(tokens=BIG), dict(cols=BIG), dict(tokens=2 ** 20, cols=2 ** 15)):
        assert call(**kw) == m.ERR_INVALID_ARG, kw
    for kw in (dict(cols=40), dict(cols=36, **none), dict(rows=40), dict(x=HALF), dict(w=ODD),
               dict(row_of=ODD), dict(entry_of=ODD), dict(offsets=ODD), dict(rc=HALF), dict(rs=HALF),
               dict(cc=HALF), dict(cs=HALF)):
        assert call(**kw) == m.ERR_ALIGNMENT, kw
    assert call(rows=0, x=None) == m.OK
    assert call(cols=0, x=None) == m.OK


def test_combine(lib):
    def call(y=P, dt=0, rows=64, cols=64, tokens=4, k=2, w=P, row_of=P, out=P):
        return lib.mxfp8_combine(y, dt, rows, cols, tokens, k, w, row_of, out, None)

    for kw in (dict(y=None), dict(dt=7), dict(rows=-32), dict(cols=-1), dict(tokens=-1),
               dict(k=0), dict(row_of=None), dict(out=None), dict(tokens=BIG)):
        assert call(**kw) == m.ERR_INVALID_ARG, kw
    for kw in (dict(y=HALF), dict(w=ODD), dict(row_of=ODD), dict(out=HALF), dict(rows=63)):
        assert call(**kw) == m.ERR_ALIGNMENT, kw
    assert call(tokens=0, out=None, row_of=None) == m.OK
    assert call(cols=0, out=None) == m.OK


def test_combine_backward(lib):
    def call(g=P, y=P, dt=0, tokens=4, cols=64, k=2, w=P, row_of=P, entry_of=P, rows=64, gy=P,
             gw=P):
        return lib.mxfp8_combine_backward(g, y, dt, tokens, cols, k, w, row_of, entry_of, rows,
                                          gy, gw, None)

    for kw in (dict(g=None), dict(y=None), dict(dt=-1), dict(tokens=-1), dict(cols=-1),
               dict(k=0), dict(w=None), dict(row_of=None), dict(entry_of=None), dict(rows=-64),
               dict(gw=None)):
        assert call(**kw) == m.ERR_INVALID_ARG, kw
    for kw in (dict(g=HALF), dict(y=HALF), dict(w=ODD), dict(row_of=ODD), dict(entry_of=ODD),
               dict(gy=HALF), dict(gw=ODD), dict(rows=1)):
        assert call(**kw) == m.ERR_ALIGNMENT, kw
    assert call(tokens=0, rows=0, g=None, y=None, w=None, row_of=None, gw=None) == m.OK
    assert call(tokens=0, gy=None, entry_of=None) == m.OK


def test_swiglu(lib):
    def call(x=P, rows=4, width=64, h=P, codes=P, scales=P, rule=1):
        return lib.mxfp8_swiglu(x, rows, width, h, codes, scales, rule, None)

    for kw in (dict(x=None), dict(rows=-1), dict(width=-32), dict(h=None), dict(codes=None),
               dict(scales=None), dict(rule=2), dict(rows=BIG), dict(width=2 ** 31)):
        assert call(**kw) == m.ERR_INVALID_ARG, kw
    for kw in (dict(width=48), dict(x=HALF), dict(h=HALF), dict(codes=HALF)):
        assert call(**kw) == m.ERR_ALIGNMENT, kw
    assert call(rows=0, x=None, h=None) == m.OK
    assert call(width=0, x=None, h=None) == m.OK


def test_swiglu_backward(lib):
    def call(g=P, codes=P, scales=P, rows=4, width=64, gx=P, h=P):
        return lib.mxfp8_swiglu_backward(g, codes, scales, rows, width, gx, h, None)

    for kw in (dict(g=None), dict(codes=None), dict(scales=None), dict(rows=-1),
               dict(width=-32), dict(gx=None), dict(rows=BIG)):
        assert call(**kw) == m.ERR_INVALID_ARG, kw
    for kw in (dict(width=33), dict(g=HALF), dict(codes=HALF), dict(gx=HALF), dict(h=HALF)):
        assert call(**kw) == m.ERR_ALIGNMENT, kw
    assert call(rows=0, g=None, codes=None, scales=None, gx=None) == m.OK


def test_python_refuses_host_tensors():
    ids = torch.zeros(4, 2, dtype=torch.int64)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    plan = m.RoutePlan(*(torch.zeros(n, dtype=torch.int32) for n in (9, 8, 64)))
    for call in (lambda: m.route(ids, 8), lambda: m.dispatch(x, plan),
                 lambda: m.quantize_dispatch(x, plan), lambda: m.combine(x, plan),
                 lambda: m.combine_backward(x, x, plan, x.float()), lambda: m.swiglu(x),
                 lambda: m.swiglu_backward(x, x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="axis"):
        m.quantize_dispatch(x, plan, 2)


@pytest.mark.gpu
def test_python_refuses_other_shapes_and_types():
    __graft_entry__.build()
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    plan = m.route(z(4, 2, d=torch.int64), 8)
    rows, x, w = plan.entry_of.numel(), z(4, 64), z(4, 2, d=torch.float32)
    y = z(rows, 64)
    codes, scales = z(4, 64, d=torch.uint8), z(4, 2, d=torch.uint8)
    bad = [lambda: m.route(z(4, 2, d=torch.int32), 8), lambda: m.route(z(4, d=torch.int64), 8),
           lambda: m.route(z(4, 4, d=torch.int64)[:, ::2], 8),
           lambda: m.route(z(4, 2, d=torch.int64), 0),
           lambda: m.route(z(4, 2, d=torch.int64), 8, -32),
           lambda: m.dispatch(z(5, 64), plan), lambda: m.dispatch(z(4, 64, d=torch.float16), plan),
           lambda: m.dispatch(z(4, 128)[:, ::2], plan),
           lambda: m.dispatch(x, plan, w[:, :1].contiguous()),
           lambda: m.dispatch(x, plan, w.double()), lambda: m.dispatch(x, plan, out=z(rows, 63)),
           lambda: m.dispatch(x, plan._replace(row_of=plan.row_of.view(-1))),
           lambda: m.dispatch(x, plan._replace(entry_of=plan.entry_of.long())),
           lambda: m.quantize_dispatch(x.float(), plan),
           lambda: m.quantize_dispatch(x, plan, out=z(rows, 63, d=torch.uint8)),
           lambda: m.quantize_dispatch(x, plan, scales=z(8, d=torch.uint8)),
           lambda: m.combine(z(rows + 32, 64), plan), lambda: m.combine(y, plan, w.half()),
           lambda: m.combine(y, plan, out=z(3, 64)),
           lambda: m.combine_backward(x, y, plan, None),
           lambda: m.combine_backward(x.float(), y, plan, w),
           lambda: m.combine_backward(z(4, 32), y, plan, w),
           lambda: m.combine_backward(x, y, plan, w, grad_rows=False, out=y),
           lambda: m.combine_backward(x, y, plan, w, out_weights=w[:1]),
           lambda: m.swiglu(z(4, 96)), lambda: m.swiglu(z(4, 64, d=torch.float32)),
           lambda: m.swiglu(x, checkpoint=False, codes=codes),
           lambda: m.swiglu(x, out=z(4, 31)), lambda: m.swiglu(x, scales=z(7, d=torch.uint8)),
           lambda: m.swiglu_backward(z(4, 48), codes, scales),
           lambda: m.swiglu_backward(z(4, 32), codes[:3], scales),
           lambda: m.swiglu_backward(z(4, 32), codes, scales[:3]),
           lambda: m.swiglu_backward(z(4, 32), codes, scales, out_h=x)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    with pytest.raises(m.MXFP8Error):
        m.route(z(4, 2, d=torch.int64), 8, 100)
    with pytest.raises(m.MXFP8Error):
        m.swiglu(x, rule=5)
    assert m.device_status() == m.OK
