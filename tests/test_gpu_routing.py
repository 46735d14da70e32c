"""GPU parity of expert routing (the plan, rows to the segments and back, gradients) against
the CPU oracle.

Tolerances. A dispatched row is one FP32 product rounded to its type: compared bit for bit with
the same two roundings on the CPU. combine adds k FP32 products in order: each of the k fused steps
rounds a partial sum that is at most sum |w y|, so FP32 is off by at most (k + 1) 2^-24 sum |w y|;
BF16 results add half a step, 2^-8 of the result. A weight's gradient is a sum of `cols`
products: a thread adds at most cols / 128 + 128 of them, then at most 16 joins follow:
(cols / 128 + 144) 2^-24 sum |g y|."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle.mxfp8_oracle as O
import oracle.routing_oracle as R
from tests.oracle_helpers import bf16_bits, gpu_ready, u8

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def m():
    mod = gpu_ready()
    yield mod
    assert mod.device_status() == mod.OK


def choices(seed, tokens, k, experts, dropped=0.0, skew=1.0):
    """int64 [tokens, k], popular experts first, the same expert twice now and then."""
    g = np.random.default_rng(seed)
    p = (1.0 + np.arange(experts)) ** -skew
    ids = g.choice(experts, (tokens, k), p=p / p.sum())
    ids = g.permutation(experts)[ids]
    ids[g.random((tokens, k)) < dropped] = -1
    return torch.from_numpy(ids.astype(np.int64))


def want_plan(ids, experts, rows):
    return [torch.from_numpy(a.astype(np.int32)) for a in R.route(ids.numpy(), experts, rows)]


def check_plan(m, ids, experts, rows=None):
    plan = m.route(ids.to(DEV), experts, rows)
    rows = R.rows_for(*ids.shape, experts) if rows is None else rows
    for name, got, want in zip(plan._fields, plan, want_plan(ids, experts, rows)):
        assert got.dtype == torch.int32
        np.testing.assert_array_equal(got.cpu().numpy(), want.numpy(), err_msg=name)
    return plan


@pytest.mark.parametrize("tokens,k,experts,dropped", [
    (0, 2, 4, 0.0), (1, 1, 1, 0.0), (1, 8, 128, 0.0), (1, 8, 128, 1.0), (5, 3, 2, 0.3),
    (37, 8, 128, 0.0), (33, 1, 1024, 0.1), (509, 6, 60, 0.1), (700, 6, 1000, 0.0),
    (1021, 8, 8, 0.5), (4096, 2, 16, 0.0), (4099, 4, 256, 0.2), (8192, 8, 128, 0.0),
    (30011, 7, 1024, 0.1), (131072, 8, 64, 0.0), (16400, 8, 100, 0.0),
    (150001, 8, 1000, 0.1)]
    # every size of the kernel's shared memory: runs of 32 to 512 entries a warp
    + [(8 * 32 * 32 * n // 4, 4, e, 0.02) for n in range(1, 34) for e in (16, 130)])
def test_route(m, tokens, k, experts, dropped):
    check_plan(m, choices(tokens + k, tokens, k, experts, dropped), experts)


@pytest.mark.parametrize("tokens", [1, 31, 32, 33, 256, 257, 5000, 70000])
def test_route_one_expert_takes_all(m, tokens):
    check_plan(m, torch.full((tokens, 1), 3, dtype=torch.int64), 4)
    check_plan(m, torch.full((tokens, 1), -5, dtype=torch.int64), 4)


def test_route_exact_rows(m):
    ids = choices(3, 200, 2, 7, 0.1)
    need = sum(-(-int((ids == e).sum()) // 32) * 32 for e in range(7))
    check_plan(m, ids, 7, need)
    check_plan(m, ids, 7, need + 32)
    check_plan(m, torch.full((9, 2), -1, dtype=torch.int64), 7, 0)


def test_route_too_few_rows_is_latched(m):
    ids = choices(4, 200, 2, 7)
    check_plan(m, ids, 7, 128)
    assert m.device_status() == m.ERR_BAD_OFFSETS
    check_plan(m, choices(4, 9000, 8, 60), 60, 32)
    assert m.device_status() == m.ERR_BAD_OFFSETS


@pytest.mark.parametrize("bad", [7, 8, 2 ** 31, 2 ** 32 + 1, 2 ** 62])
def test_route_bad_expert_is_latched(m, bad):
    ids = choices(5, 3000, 4, 7, 0.1)
    with_bad = ids.clone()
    with_bad[1234, 2] = bad
    ids[1234, 2] = -1
    plan = m.route(with_bad.to(DEV), 7)
    assert m.device_status() == m.ERR_BAD_EXPERT
    for got, want in zip(plan, want_plan(ids, 7, R.rows_for(3000, 4, 7))):
        np.testing.assert_array_equal(got.cpu().numpy(), want.numpy())


def values(seed, rows, cols, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(rows, cols, generator=g).to(dtype)


def weights(seed, tokens, k):
    return torch.rand(tokens, k, generator=torch.Generator().manual_seed(seed))


SIZES = [(1, 8, 128, 2048, 0.0), (70, 2, 6, 4098, 0.1), (70, 1, 6, 1030, 0.0), (50, 3, 9, 2052, 0.0),
         (40, 2, 4, 8192, 0.1), (90, 4, 4, 516, 0.0), (37, 3, 5, 1, 0.0), (33, 2, 4, 7, 0.2), (60, 1, 3, 8, 0.0),
         (129, 8, 16, 1033, 0.1), (257, 4, 8, 136, 0.5), (65, 40, 12, 72, 0.1), (7, 2, 3, 4104, 1.0),
         (301, 6, 60, 513, 0.0)]


def guarded(rows, cols, dtype):
    """A buffer with a margin behind it, filled with a value that no result has."""
    buf = torch.full((rows * cols + 64,), -77.0, dtype=dtype, device=DEV)
    return buf[:rows * cols].view(rows, cols), buf[rows * cols:]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("tokens,k,experts,cols,dropped", SIZES)
def test_dispatch(m, tokens, k, experts, cols, dropped, weighted, dtype):
    ids = choices(tokens, tokens, k, experts, dropped)
    plan = check_plan(m, ids, experts)
    rows = plan.entry_of.numel()
    x = values(1, tokens, cols, dtype)
    w = weights(2, tokens, k) if weighted else None
    out, margin = guarded(rows, cols, dtype)
    m.dispatch(x.to(DEV), plan, None if w is None else w.to(DEV), out=out)
    entry = plan.entry_of.cpu().long()
    want = x[entry.clamp(min=0) // k]
    if weighted:
        want = (want.float() * w.view(-1)[entry.clamp(min=0)][:, None]).to(dtype)
    want[entry < 0] = 0
    assert torch.equal(out.cpu(), want)
    assert (margin == -77).all()


def combine_close(got, want, mag, k, dtype):
    tol = (k + 1) * 2.0 ** -24 * mag
    if dtype == BF16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want) + 2.0 ** -133
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol + 2.0 ** -148).all(), np.max(err - tol)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("tokens,k,experts,cols,dropped", SIZES)
def test_combine(m, tokens, k, experts, cols, dropped, weighted, dtype):
    plan = m.route(choices(tokens, tokens, k, experts, dropped).to(DEV), experts)
    y = values(3, plan.entry_of.numel(), cols, dtype)
    y[plan.entry_of.cpu() < 0] = float("nan")          # padding rows are not read
    w = weights(4, tokens, k) if weighted else None
    out, margin = guarded(tokens, cols, dtype)
    if weighted:    # nor are the weights of entries without a row
        w[plan.row_of.cpu() < 0] = float("nan")
    m.combine(y.to(DEV), plan, None if w is None else w.to(DEV), out=out)
    want, mag = R.combine(y.double().numpy(), plan.row_of.cpu().numpy(),
                          None if w is None else w.numpy())
    combine_close(out, want, mag, k, dtype)
    assert (margin == -77).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("tokens,k,experts,cols,dropped", SIZES)
def test_combine_backward(m, tokens, k, experts, cols, dropped, dtype):
    plan = m.route(choices(tokens, tokens, k, experts, dropped).to(DEV), experts)
    rows, row_of = plan.entry_of.numel(), plan.row_of.cpu().numpy()
    y, g, w = values(5, rows, cols, dtype), values(6, tokens, cols, dtype), weights(7, tokens, k)
    y[plan.entry_of.cpu() < 0] = float("nan")
    w[plan.row_of.cpu() < 0] = float("nan")
    out, margin = guarded(rows, cols, dtype)
    grad_y, grad_w = m.combine_backward(g.to(DEV), y.to(DEV), plan, w.to(DEV), out=out)
    assert grad_y is out and grad_w.dtype == FP32 and (margin == -77).all()
    entry = plan.entry_of.cpu().long()
    want = (g[entry.clamp(min=0) // k].float()
            * w.view(-1)[entry.clamp(min=0)][:, None]).to(dtype)
    want[entry < 0] = 0
    assert torch.equal(grad_y.cpu(), want)
    want, mag = R.combine_weights_grad(g.double().numpy(), y.double().numpy(), row_of)
    err = np.abs(grad_w.double().cpu().numpy() - want)
    assert (err <= (cols / 128 + 144) * 2.0 ** -24 * mag).all()
    # the weights' part alone, and the rows' gradient in place of y: the same bits
    none, alone = m.combine_backward(g.to(DEV), y.to(DEV), plan, w.to(DEV), grad_rows=False)
    assert none is None and torch.equal(alone, grad_w)
    inplace = y.to(DEV)
    _, again = m.combine_backward(g.to(DEV), inplace, plan, w.to(DEV), out=inplace)
    assert torch.equal(inplace, grad_y) and torch.equal(again, grad_w)


def test_gradients_are_those_of_the_sums_by_differences(m):
    """combine is linear in y and in the weights, so a difference of any length gives its
    gradients exactly, but for the roundings of the two FP32 sums."""
    tokens, k, experts, cols = 19, 3, 5, 40
    plan = m.route(choices(8, tokens, k, experts, 0.1).to(DEV), experts)
    y, g = values(9, plan.entry_of.numel(), cols, FP32), values(10, tokens, cols, FP32)
    w = weights(11, tokens, k)
    grad_y, grad_w = m.combine_backward(g.to(DEV), y.to(DEV), plan, w.to(DEV))

    def total(y_, w_):
        return (m.combine(y_.to(DEV), plan, w_.to(DEV)).double().cpu() * g.double()).sum().item()

    base = total(y, w)
    _, mag = R.combine(np.abs(y.double().numpy()) + 1, plan.row_of.cpu().numpy(), w.numpy() + 1)
    tol = 4 * (k + 1) * 2.0 ** -24 * (mag * np.abs(g.double().numpy())).sum()
    for t, j in [(0, 0), (7, 2), (18, 1)]:
        up = w.clone()
        up[t, j] += 1
        step = (up[t, j] - w[t, j]).item()
        assert abs((total(y, up) - base) / step - grad_w[t, j].item()) <= tol
        r = plan.row_of[t, j].item()
        if r >= 0:
            up = y.clone()
            up[r, 5] += 1
            step = (up[r, 5] - y[r, 5]).item()
            assert abs((total(up, w) - base) / step - grad_y[r, 5].item()) <= tol


def check_quantized(m, x, plan, experts, w):
    """quantize_dispatch of both axes and both at once: bytes of the grouped quantizer on the
    dispatched rows (the whole code buffers, and the scales against the oracle's layout)."""
    rows, cols = plan.entry_of.numel(), x.shape[1]
    off = plan.offsets.cpu().numpy()
    xd = x.to(DEV)
    wd = None if w is None else w.to(DEV)
    spread = m.dispatch(xd, plan, wd)
    bits = bf16_bits(spread)
    dual = m.quantize_dispatch_dual(xd, plan, wd)
    for axis, pair in ((m.ROW, dual[:2]), (m.COL, dual[2:])):
        codes, scales = m.quantize_dispatch(xd, plan, axis, wd)
        assert torch.equal(codes, pair[0]) and torch.equal(scales, pair[1])
        ref, _ = m.quantize_grouped(spread, plan.offsets, axis)
        assert torch.equal(codes, ref)
        want_codes, want_scales = O.quantize(bits, O.ROW if axis == m.ROW else O.COL)
        np.testing.assert_array_equal(u8(codes), want_codes)
        swizzle = O.swizzle_grouped_rows if axis == m.ROW else O.swizzle_grouped_cols
        want = swizzle(want_scales, off)
        got = u8(scales)
        assert got.size == m.grouped_scale_bytes(rows, cols, experts, axis)
        np.testing.assert_array_equal(got[:want.size], want)
        assert not got[want.size:].any()


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("tokens,k,experts,cols,dropped", [
    (1, 8, 128, 2048, 0.0), (37, 8, 16, 32, 0.0), (300, 2, 3, 96, 0.2), (129, 3, 300, 160, 0.1),
    (1021, 6, 8, 224, 0.0), (5, 1, 2, 1056, 1.0), (700, 1, 1, 128, 0.0), (60, 40, 5, 544, 0.1),
    (33, 2, 1000, 2592, 0.0), (6000, 2, 4, 256, 0.3)])
def test_quantize_dispatch(m, tokens, k, experts, cols, dropped, weighted):
    plan = m.route(choices(tokens, tokens, k, experts, dropped).to(DEV), experts)
    x = values(12, tokens, cols, BF16)
    x[:, ::17] *= 30
    check_quantized(m, x, plan, experts, weights(13, tokens, k) if weighted else None)


def test_quantize_dispatch_of_many_elements(m):
    """Each way that both copies are made, on either side of the sizes that choose between them:
    against the grouped quantizer on the dispatched rows."""
    for tokens, k, cols, weighted in ((8192, 8, 2048, False), (5000, 7, 4096, False),
                                      (8191, 8, 2048, False), (4096, 2, 2048, False),
                                      (4095, 2, 2048, False), (2048, 8, 1056, True),
                                      (1000, 8, 1056, True), (16384, 1, 1024, False)):
        plan = m.route(choices(34, tokens, k, 64, 0.0).to(DEV), 64)
        x = torch.randn(tokens, cols, device=DEV).to(BF16)
        x[17, 100:200] = float("inf")
        w = weights(35, tokens, k).to(DEV) if weighted else None
        spread = m.dispatch(x, plan, w)
        got = m.quantize_dispatch_dual(x, plan, w)
        want = m.quantize_grouped_dual(spread, plan.offsets)
        assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
        off = plan.offsets.cpu().numpy()
        tiles = int(((off[1:] - off[:-1] + 127) // 128).sum())
        for a, b, per in ((got[1], want[1], -(-cols // 128)), (got[3], want[3], -(-cols // 128))):
            assert torch.equal(a[:tiles * per * 512], b[:tiles * per * 512])
            assert not a[tiles * per * 512:].any()


@pytest.mark.parametrize("tokens,k,cols,experts,weighted", [
    (1024, 8, 2048, 128, False), (4096, 8, 2048, 128, False), (16384, 2, 1024, 64, False),
    (4096, 2, 4096, 8, True), (16384, 1, 5120, 16, True), (16384, 4, 4096, 32, False),
    (16383, 4, 4096, 32, True), (8192, 8, 4096, 3, True)])
def test_quantize_dispatch_shares(m, tokens, k, cols, experts, weighted):
    """Both copies in any share of the CTAs, and in turn, are the bytes of each alone."""
    plan = m.route(choices(36, tokens, k, experts, 0.1).to(DEV), experts)
    x = torch.randn(tokens, cols, device=DEV).to(BF16)
    w = weights(37, tokens, k).to(DEV) if weighted else None
    got = m.quantize_dispatch_dual(x, plan, w)
    for a, b in zip(got, (*m.quantize_dispatch(x, plan, m.ROW, w),
                          *m.quantize_dispatch(x, plan, m.COL, w))):
        assert torch.equal(a, b)


@pytest.mark.parametrize("tokens,k,weighted", [
    (4096, 40, True), (30000, 40, True), (30000, 40, False), (30000, 1, True), (3, 1000, True)])
def test_quantize_dispatch_of_few_rows_of_many_entries(m, tokens, k, weighted):
    """Nearly all entries of no expert, and no more rows than the others need: both copies are
    written whole."""
    ids = torch.full((tokens, k), -1, dtype=torch.int64)
    ids[::tokens // 3, 0] = 1
    plan = m.route(ids.to(DEV), 2, rows=32)
    x = values(38, tokens, 96, BF16).to(DEV)
    w = weights(39, tokens, k).to(DEV) if weighted else None
    bytes_ = [torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV) for n in
              (32 * 96, m.grouped_scale_bytes(32, 96, 2, m.ROW),
               32 * 96, m.grouped_scale_bytes(32, 96, 2, m.COL))]
    m.quantize_dispatch_dual(x, plan, w, *bytes_)
    for got, want in zip(bytes_, (*m.quantize_dispatch(x, plan, m.ROW, w),
                                  *m.quantize_dispatch(x, plan, m.COL, w))):
        assert torch.equal(got, want.flatten())
    assert m.device_status() == m.OK


def test_quantize_dispatch_of_nan_infinity_and_tiny_values(m):
    tokens, k, experts, cols = 200, 2, 4, 128
    plan = m.route(choices(14, tokens, k, experts).to(DEV), experts)
    x = values(15, tokens, cols, BF16)
    x[3, 5], x[50, 70], x[90, 1] = float("nan"), float("inf"), -float("inf")
    x[100:110] = 2.0 ** -130
    x[120] = 0
    check_quantized(m, x, plan, experts, None)
    check_quantized(m, x, plan, experts, weights(16, tokens, k))


def test_quantize_dispatch_of_every_magnitude(m):
    """Rows and weights over the exponents of their types, subnormals, zeros, infinities and NaN
    among the weights; within a row values down to 2^-20 of the largest."""
    tokens, k, experts, cols = 3000, 5, 4, 96
    g = torch.Generator().manual_seed(41)
    plan = m.route(choices(42, tokens, k, experts, 0.1).to(DEV), experts)
    rand = lambda *n: torch.rand(*n, generator=g, dtype=torch.float64)  # noqa: E731
    sign = lambda *n: torch.where(rand(*n) < 0.5, -1.0, 1.0).double()  # noqa: E731
    level = torch.floor(rand(tokens, 1) * 266 - 138) - torch.floor(rand(tokens, cols) * 21)
    x = (sign(tokens, cols) * (1 + rand(tokens, cols)) * 2.0 ** level).to(BF16)
    x[torch.isinf(x)] = 1.5
    w = (sign(tokens, k) * (1 + rand(tokens, k))
         * 2.0 ** torch.floor(rand(tokens, k) * 276 - 149)).float()
    w[::2] = (sign(1500, k) * (1 + rand(1500, k)) * 2.0 ** torch.floor(
        rand(1500, k) * 40 - 20 - level[::2].max(1, keepdim=True).values.clamp(-100, 100))).float()
    w[7, 0], w[9, 1], w[11, 2], w[13, 3] = 0.0, -0.0, float("inf"), float("nan")
    check_quantized(m, x, plan, experts, w)


def test_quantize_dispatch_column_copy_of_a_narrow_width(m):
    """The column copy alone takes any multiple of 8 columns."""
    plan = m.route(choices(17, 90, 2, 4).to(DEV), 4)
    x = values(18, 90, 40, BF16).to(DEV)
    codes, scales = m.quantize_dispatch(x, plan, m.COL)
    want, want_scales = m.quantize_grouped(m.dispatch(x, plan), plan.offsets, m.COL)
    assert torch.equal(codes, want)
    used = O.swizzle_grouped_cols(O.quantize(bf16_bits(m.dispatch(x, plan)), O.COL)[1],
                                  plan.offsets.cpu().numpy()).size
    assert torch.equal(scales[:used], want_scales[:used])


def test_quantize_dispatch_bad_offsets_are_latched(m):
    plan = m.route(choices(19, 64, 2, 4).to(DEV), 4)
    offsets = plan.offsets.clone()
    offsets[1] += 1
    codes = torch.full((plan.entry_of.numel(), 64), 99, dtype=torch.uint8, device=DEV)
    m.quantize_dispatch(values(20, 64, 64, BF16).to(DEV), plan._replace(offsets=offsets), m.ROW,
                        out=codes)
    assert m.device_status() == m.ERR_BAD_OFFSETS
    assert (codes == 99).all()


def test_a_plan_of_other_rows_is_not_followed(m):
    """Rows past the segments, entries past the tokens: latched and skipped."""
    plan = m.route(choices(21, 64, 2, 4).to(DEV), 4)
    x = values(22, 64, 64, BF16).to(DEV)
    y = values(23, plan.entry_of.numel(), 64, BF16).to(DEV)
    w = weights(24, 64, 2).to(DEV)
    rows = plan.entry_of.numel()
    row_of, entry_of = plan.row_of.clone(), plan.entry_of.clone()
    row_of[5, 1] = rows
    entry_of[0] = 128
    wrong = plan._replace(row_of=row_of, entry_of=entry_of)
    right = row_of.clone()
    right[5, 1] = -1
    right = plan._replace(row_of=right)
    for call in (lambda p: m.combine(y, p, w), lambda p: m.combine_backward(x, y, p, w)[1]):
        got = call(wrong)
        assert m.device_status() == m.ERR_BAD_OFFSETS
        assert torch.equal(got, call(right))
    m.dispatch(x, wrong)
    assert m.device_status() == m.ERR_BAD_OFFSETS
    m.quantize_dispatch(x, wrong)
    assert m.device_status() == m.ERR_BAD_OFFSETS
    codes, _ = m.quantize_dispatch(x, wrong, m.COL)
    assert m.device_status() == m.ERR_BAD_OFFSETS
    assert not codes[:, 0].any()


def test_no_tokens(m):
    ids = torch.empty(0, 2, dtype=torch.int64, device=DEV)
    plan = m.route(ids, 3, 64)
    assert plan.offsets.tolist() == [0, 0, 0, 64]
    x = torch.empty(0, 96, dtype=BF16, device=DEV)
    w = torch.empty(0, 2, device=DEV)
    assert not m.dispatch(x, plan).any()
    codes, scales = m.quantize_dispatch(x, plan)
    assert not codes.any() and not scales.any()
    y = torch.ones(64, 96, dtype=BF16, device=DEV)
    assert m.combine(y, plan).shape == (0, 96)
    grad_y, grad_w = m.combine_backward(x, y, plan, w)
    assert not grad_y.any() and grad_w.shape == (0, 2)
    empty = m.route(ids, 3)
    assert empty.entry_of.numel() == 0 and m.dispatch(x, empty).shape == (0, 96)
    assert m.quantize_dispatch_dual(x, empty)[0].shape == (0, 96)
    some = m.route(torch.full((4, 2), -1, dtype=torch.int64, device=DEV), 3, 0)
    none = torch.empty(0, 96, dtype=BF16, device=DEV)
    assert not m.combine(none, some).any()
    ones = torch.ones(4, 96, dtype=BF16, device=DEV)
    grad_y, grad_w = m.combine_backward(ones, none, some, torch.ones(4, 2, device=DEV))
    assert grad_y.shape == (0, 96) and not grad_w.any()
    no_cols = m.combine_backward(ones[:, :0].contiguous(), none[:, :0].contiguous(), some,
                                 torch.ones(4, 2, device=DEV))
    assert not no_cols[1].any()


@pytest.mark.parametrize("tokens,k,experts,cols", [(300, 4, 12, 160), (9000, 8, 128, 64)])
def test_captured_and_replayed_on_new_choices(m, tokens, k, experts, cols):
    ids = choices(25, tokens, k, experts).to(DEV)
    x, w = values(26, tokens, cols, BF16).to(DEV), weights(27, tokens, k).to(DEV)

    def step():
        plan = m.route(ids, experts)
        y = m.dispatch(x, plan, w)
        q = m.quantize_dispatch_dual(x, plan)
        out = m.combine(y, plan, w)
        return (*plan, y, *q, out, *m.combine_backward(x, y, plan, w))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            held = step()
    for seed in (28, 29):
        ids.copy_(choices(seed, tokens, k, experts, 0.2))
        x.copy_(values(seed, tokens, cols, BF16))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, step()):
            assert torch.equal(a, b)


def test_launches_back_to_back_keep_their_order(m):
    """Each launch reads what the one before wrote, and overwrites what the one before read, with no
    host synchronization between; and again without programmatic launches, in a child process."""
    tokens, k, experts, cols = 2000, 4, 12, 96
    ids = [choices(40 + i, tokens, k, experts, 0.1).to(DEV) for i in range(4)]
    w = weights(44, tokens, k).to(DEV)
    x0 = values(45, tokens, cols, BF16).to(DEV)

    def chain(wait):
        x, sums = x0.clone(), []
        rows = R.rows_for(tokens, k, experts)
        y = torch.empty(rows, cols, dtype=BF16, device=DEV)
        for i in range(12):
            plan = m.route(ids[i % 4], experts)
            wait()
            m.dispatch(x, plan, w, out=y)
            wait()
            sums.append(m.quantize_dispatch_dual(x, plan)[0].clone())
            wait()
            m.combine(y, plan, w, out=x)
            wait()
            m.combine_backward(x, y, plan, w, out=y)
            wait()
            m.combine(y, plan, out=x)
            wait()
        return [x] + sums

    for a, b in zip(chain(lambda: None), chain(torch.cuda.synchronize)):
        assert torch.equal(a, b)


def test_without_programmatic_launches():
    r = subprocess.run(
        [sys.executable, "-m", "pytest", "-q", "-x", __file__, "-k", "order or captured or another"],
        env=dict(os.environ, MXFP8_PDL="0"), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:]


def test_on_another_stream(m):
    tokens, k, experts, cols = 513, 4, 12, 160
    ids = choices(30, tokens, k, experts).to(DEV)
    x, w = values(31, tokens, cols, BF16).to(DEV), weights(32, tokens, k).to(DEV)
    plan = m.route(ids, experts)
    y = m.dispatch(x, plan, w)
    want = (*plan, y, *m.quantize_dispatch_dual(x, plan, w), m.combine(y, plan, w),
            *m.combine_backward(x, y, plan, w))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p = m.route(ids, experts, stream=side)
    y2 = m.dispatch(x, p, w, stream=side)
    got = (*p, y2, *m.quantize_dispatch_dual(x, p, w, stream=side),
           m.combine(y2, p, w, stream=side), *m.combine_backward(x, y2, p, w, stream=side))
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_rows_past_two_to_the_31_elements(m):
    """Offsets of rows need 64 bits: 66000 rows and more of 33000 columns."""
    tokens, cols = 66000, 33000
    ids = choices(33, tokens, 1, 2).to(DEV)
    plan = m.route(ids, 2)
    rows = plan.entry_of.numel()
    assert rows * cols > 2 ** 31
    x = torch.zeros(tokens, cols, dtype=BF16, device=DEV)
    x[:, -1] = torch.arange(tokens, device=DEV) % 251
    x[:, 0] = torch.arange(tokens, device=DEV) % 127
    y = m.dispatch(x, plan)
    entry = plan.entry_of.long()
    for c in (0, cols - 1):
        want = torch.where(entry < 0, 0.0, x[:, c][entry.clamp(min=0)].float())
        assert torch.equal(y[:, c].float(), want)
    assert torch.equal(m.combine(y, plan), x)
    w = torch.full((tokens, 1), 2.0, device=DEV)
    grad_w = m.combine_backward(x, y, plan, w, out=y)[1]
    assert torch.equal(grad_w[:, 0], x[:, 0].float() ** 2 + x[:, -1].float() ** 2)
    assert torch.equal(y[:, -1].float(),
                       2 * torch.where(entry < 0, 0.0, x[:, -1][entry.clamp(min=0)].float()))


def test_quantize_dispatch_past_two_to_the_31_bytes(m):
    """Both copies of 66000 rows and more of 33024 columns: the grouped quantizer's."""
    tokens, k, cols, experts = 33000, 2, 33024, 3
    plan = m.route(choices(40, tokens, k, experts).to(DEV), experts)
    assert plan.entry_of.numel() * cols > 2 ** 31
    x = torch.randn(tokens, cols, device=DEV, dtype=BF16)
    got = m.quantize_dispatch_dual(x, plan)
    want = m.quantize_grouped_dual(m.dispatch(x, plan), plan.offsets)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    off = plan.offsets.cpu()
    used = int(((off[1:] - off[:-1] + 127) // 128).sum()) * (cols // 128) * 512
    for a, b in ((got[1], want[1]), (got[3], want[3])):
        assert torch.equal(a[:used], b[:used]) and not a[used:].any()
