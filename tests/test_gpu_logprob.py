"""GPU parity of token log probabilities, entropy, likeliest tokens and their gradient
against the float64 oracle.

Tolerances: a log probability is d_t - log S with d = (x - m) / T. d carries two FP32
roundings. S is a sum of positive terms: each term is off by 2^-22 (ex2) plus the rounding of
its exponent, and a thread adds up to `chain` of them in order, then a few more steps join
the threads: |error of log S| <= (chain + 64) 2^-24 + 2^-20. The entropy adds a second such
sum, of weight up to the entropy itself. p_v is 2^t with t = log2 p_v rounded three times."""
import numpy as np
import pytest
import torch

import oracle.logprob_oracle as L
from tests.oracle_helpers import gpu_ready

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF = float("inf")


@pytest.fixture(scope="module")
def m():
    mod = gpu_ready()
    yield mod
    assert mod.device_status() == mod.OK


def log_sum_error(vocab):
    chain = -(-vocab // 256) + 8       # values one thread adds, at most
    return (chain + 64) * 2.0 ** -24 + 2.0 ** -20


def close(got, want, tol):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    fine = np.isfinite(want)
    np.testing.assert_array_equal(got[~fine], want[~fine])      # NaN and infinities
    err = np.abs(got[fine] - want[fine])
    tol = np.broadcast_to(tol, want.shape)[fine]
    assert np.all(err <= tol), f"worst {np.max(err - tol)}"


def make(seed, rows, vocab, dtype, pitch=None, offset=0, sigma=3.0):
    """Logits [rows, vocab] of any row pitch and start, targets, float64 copies."""
    g = torch.Generator().manual_seed(seed)
    pitch = vocab if pitch is None else pitch
    buf = torch.full((rows * pitch + offset + 8,), float("nan"), dtype=dtype, device=DEV)
    x = buf[offset:offset + rows * pitch].view(rows, pitch)[:, :vocab]
    x.copy_((torch.randn(rows, vocab, generator=g) * sigma).to(dtype))
    t = torch.randint(vocab, (rows,), generator=g)
    t[torch.rand(rows, generator=g) < 0.2] = -1
    return x, t.to(DEV)


def check_forward(m, x, t, temperature, top):
    r = m.token_logprobs(x, t, temperature, top)
    xs = x.double().cpu().numpy()
    want = L.forward(xs, t.cpu().numpy(), temperature, top)
    err = log_sum_error(xs.shape[1])
    with np.errstate(invalid="ignore"):
        lp_tol = err + np.abs(want["logprob"]) * 2.0 ** -22
        close(r.logprob.cpu(), want["logprob"], lp_tol)
        h = want["entropy"]
        close(r.entropy.cpu(), h, 2 * err * (2 + np.abs(h)))
        close(r.stats.cpu(), want["stats"], err)
    if top:
        np.testing.assert_array_equal(r.top_id.cpu().numpy(), want["top_id"])
        with np.errstate(invalid="ignore"):
            close(r.top_logprob.cpu(), want["top_logprob"],
                  err + np.abs(want["top_logprob"]) * 2.0 ** -22)
    else:
        assert r.top_id is None and r.top_logprob is None
    return r


def check_backward(m, x, t, temperature, top, seed=0, entropy=True, out=None):
    r = m.token_logprobs(x, t, temperature, top)
    g = np.random.default_rng(seed)
    rows, vocab = x.shape
    gl = g.standard_normal(rows).astype(np.float32)
    ge = g.standard_normal(rows).astype(np.float32) if entropy else None
    gt = g.standard_normal((rows, top)).astype(np.float32) if top else None
    xs, ts = x.double().cpu().numpy(), t.cpu().numpy()
    ids = r.top_id.cpu().numpy() if top else None
    want = L.backward(xs, ts, temperature, gl, ge, ids, gt)
    dev = lambda a: None if a is None else torch.from_numpy(a).to(DEV)  # noqa: E731
    got = m.token_logprobs_backward(x, t, r.stats, r.entropy, dev(gl), dev(ge), r.top_id,
                                    dev(gt), temperature, out=out)
    assert got.shape == x.shape and got.dtype == x.dtype
    # |p_v| times the size of its factor, and the relative error of both
    peak = np.max(xs, axis=1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        d = np.where(np.isfinite(peak), (xs - peak) / temperature, -np.inf)
        s = np.exp(d).sum(axis=1, keepdims=True)
        p = np.where(s > 0, np.exp(d) / s, 0.0)
        logp = np.where(p > 0, np.log(p), 0.0)
    size = np.abs(gl)[:, None] + (np.abs(gt).sum(1, keepdims=True) if top else 0)
    if entropy:
        size = size + np.abs(ge)[:, None] * (1 + np.abs(logp) + np.log(vocab))
    err = log_sum_error(vocab)
    tol = p * size / temperature * (2 * err + (np.abs(logp) + 4) * 2.0 ** -22) + 1e-36
    # the named columns: a sum of a few terms of either sign
    size = np.broadcast_to(size, want.shape)
    for named in (ts[:, None], ids) if top else (ts[:, None],):
        for i, c in np.argwhere(named >= 0):
            tol[i, named[i, c]] += size[i, named[i, c]] / temperature * 2.0 ** -20
    if x.dtype == torch.bfloat16:
        tol = tol + np.abs(want) * 2.0 ** -8
    close(got.double().cpu(), want, tol)
    return got


SHAPES = [(1, 1), (1, 7), (2, 8), (3, 33), (5, 256), (4, 1000), (2, 4099), (9, 8192),
          (1, 50021), (3, 131072), (400, 517)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("top", [0, 1, 5, 32])
def test_forward(m, shape, dtype, top):
    x, t = make(shape[0] + shape[1], *shape, dtype)
    check_forward(m, x, t, 1.0, top)


@pytest.mark.parametrize("pitch,offset", [(1000, 0), (1000, 1), (1001, 0), (1003, 5), (1016, 3),
                                          (1024, 8)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_any_row_pitch_and_alignment(m, pitch, offset, dtype):
    x, t = make(pitch + offset, 6, 997, dtype, pitch, offset)
    check_forward(m, x, t, 0.7, 8)
    check_backward(m, x, t, 0.7, 8)
    # a result of another pitch and alignment than the logits'
    buf = torch.full((6 * 1007 + 8,), 5.0, dtype=dtype, device=DEV)
    out = buf[3:3 + 6 * 1007].view(6, 1007)[:, :997]
    check_backward(m, x, t, 0.7, 8, out=out)
    rest = buf[3:3 + 6 * 1007].view(6, 1007)[:, 997:]
    assert (rest == 5.0).all() and (buf[:3] == 5.0).all() and (buf[3 + 6 * 1007:] == 5.0).all()


@pytest.mark.parametrize("temperature", [0.05, 0.6, 1.0, 7.0])
def test_temperature(m, temperature):
    x, t = make(11, 20, 3001, torch.float32)
    check_forward(m, x, t, temperature, 4)
    check_backward(m, x, t, temperature, 4)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("top,entropy", [(0, False), (0, True), (6, True)])
def test_backward(m, shape, dtype, top, entropy):
    x, t = make(shape[0] * 3 + shape[1], *shape, dtype)
    check_backward(m, x, t, 1.0, top, entropy=entropy)


def test_gradient_against_differences(m):
    """The GPU gradient along random directions against central differences of the float64
    forward."""
    x, t = make(5, 8, 301, torch.float32)
    r = m.token_logprobs(x, t, 0.8, 3)
    g = np.random.default_rng(4)
    gl, ge, gt = (g.standard_normal(s).astype(np.float32) for s in (8, 8, (8, 3)))
    dev = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    dx = m.token_logprobs_backward(x, t, r.stats, r.entropy, dev(gl), dev(ge), r.top_id, dev(gt),
                                   0.8).double().cpu().numpy()
    xs, ts, ids = x.double().cpu().numpy(), t.cpu().numpy(), r.top_id.cpu().numpy()

    def loss(z):
        total = np.zeros(8)
        for i in range(8):
            lp = z[i] / 0.8 - np.log(np.exp((z[i] - z[i].max()) / 0.8).sum()) - z[i].max() / 0.8
            total[i] = -ge[i] * np.sum(np.exp(lp) * lp) + np.sum(gt[i] * lp[ids[i]])
            if ts[i] >= 0:
                total[i] += gl[i] * lp[ts[i]]
        return total

    for _ in range(5):
        v = g.standard_normal(xs.shape)
        eps = 1e-5     # differences err by eps^2 times third derivatives: below 1e-8
        want = (loss(xs + eps * v) - loss(xs - eps * v)) / (2 * eps)
        assert np.all(np.abs((dx * v).sum(axis=1) - want) <= 2e-5 * (1 + np.abs(want)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masks_and_empty_rows(m, dtype):
    x, t = make(2, 12, 1203, dtype)
    lowest = torch.finfo(dtype).min
    x[0, 5:] = -INF                       # few left
    x[1, 1:] = -INF                       # one left
    x[2] = -INF                           # none left, scored
    x[3] = -INF                           # none left, not scored
    x[4, ::2] = lowest
    x[5] = lowest                         # all at the type's lowest value: uniform
    x[6, 7] = -INF
    x[7, :-3] = lowest
    x[8, 100:] = -INF
    x[8, :100] = lowest
    t[:] = torch.tensor([3, 0, 4, -1, 1, 9, 7, 0, 150, 1202, -1, 600], device=DEV)
    for temperature in (0.5, 1.0):
        check_forward(m, x, t, temperature, 8)
        check_backward(m, x, t, temperature, 8)
    r = m.token_logprobs(x, t, top=8)
    assert r.logprob[2] == -INF and r.logprob[3] == 0 and r.entropy[2] == 0
    assert (r.top_id[2] == -1).all() and (r.top_id[1, 1:] == -1).all()
    g = torch.ones(12, device=DEV)
    dx = m.token_logprobs_backward(x, t, r.stats, r.entropy, g, g)
    assert (dx[2] == 0).all() and (dx[3] == 0).all()


@pytest.mark.parametrize("rows", [3, 700])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nan_and_infinity(m, rows, dtype):
    x, t = make(3, rows, 2050, dtype)
    t[:] = 5
    x[0, 2000] = float("nan")
    x[1, 3] = INF
    r = check_forward(m, x, t, 1.0, 4)
    assert r.logprob[:2].isnan().all() and (r.top_id[:2] == -1).all()
    assert not r.logprob[2:].isnan().any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,vocab", [(1, 40000), (1, 300), (310, 3001)])
def test_ties_go_to_the_lowest_token(m, dtype, rows, vocab):
    g = torch.Generator().manual_seed(1)
    x = torch.randint(0, 3, (rows, vocab), generator=g).to(dtype).to(DEV)
    x[0] = 1.0                                           # all equal
    if rows > 2:
        x[1] = torch.arange(vocab, device=DEV).to(dtype)     # rising
        x[2] = -torch.arange(vocab, device=DEV).to(dtype)    # falling; 0 and -0
        x[2, 17] = 0.0
    t = torch.zeros(rows, dtype=torch.int64, device=DEV)
    check_forward(m, x, t, 1.0, 32)


def test_large_logits_keep_their_differences(m):
    x, t = make(8, 6, 5000, torch.float32, sigma=1.0)
    x += torch.tensor([[1e4], [-1e4], [3e5], [0], [-3e5], [1e6]], device=DEV)
    check_forward(m, x, t, 1.0, 3)
    check_backward(m, x, t, 1.0, 3)


def test_in_place_gradient(m):
    for dtype in (torch.bfloat16, torch.float32):
        x, t = make(4, 33, 2999, dtype, 3010)
        r = m.token_logprobs(x, t, 1.0, 5)
        g = torch.randn(33, device=DEV)
        gt = torch.randn(33, 5, device=DEV)
        want = m.token_logprobs_backward(x, t, r.stats, r.entropy, g, g, r.top_id, gt)
        got = m.token_logprobs_backward(x, t, r.stats, r.entropy, g, g, r.top_id, gt, out=x)
        assert got.data_ptr() == x.data_ptr() and torch.equal(got, want)


def test_same_bits_every_time_and_in_a_graph(m):
    x, t = make(6, 3, 70001, torch.bfloat16)
    want = m.token_logprobs(x, t, 0.9, 20)
    for _ in range(3):
        for a, b in zip(m.token_logprobs(x, t, 0.9, 20), want):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = m.token_logprobs(x, t, 0.9, 20)
    graph.replay()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = m.token_logprobs(x, t, 0.9, 20, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_offsets_past_32_bits(m):
    """Rows that start beyond 2^31 elements of the logits."""
    rows, vocab, pitch = 3, 1000, 1 << 30
    buf = torch.empty(2 * pitch + 1024, dtype=torch.bfloat16, device=DEV)
    x = buf.as_strided((rows, vocab), (pitch, 1))
    x.copy_(torch.randn(rows, vocab, device=DEV) * 2)
    t = torch.tensor([1, 999, 500], device=DEV)
    check_forward(m, x, t, 1.0, 3)
    r = m.token_logprobs(x, t)
    g = torch.ones(rows, device=DEV)
    got = m.token_logprobs_backward(x, t, r.stats, r.entropy, g, out=x)
    assert (got.double().sum(dim=1).abs() < 0.02).all()      # a row's gradient sums to zero


def test_target_past_the_vocabulary(m):
    x, t = make(7, 4, 100, torch.float32)
    t[:] = torch.tensor([3, 100, -5, 99], device=DEV)
    r = m.token_logprobs(x, t)
    assert m.device_status() == m.ERR_BAD_TARGET
    assert r.logprob.isnan().tolist() == [False, True, False, False] and r.logprob[2] == 0
    m.token_logprobs_backward(x, t, r.stats, r.entropy, torch.ones(4, device=DEV))
    assert m.device_status() == m.ERR_BAD_TARGET


def test_no_rows(m):
    x = torch.empty((0, 10), device=DEV)
    t = torch.empty(0, dtype=torch.int64, device=DEV)
    r = m.token_logprobs(x, t, top=3)
    assert r.logprob.shape == (0,) and r.top_id.shape == (0, 3)
    assert m.token_logprobs_backward(x, t, r.stats, r.entropy, r.logprob).shape == (0, 10)


def test_refusals(m):
    x, t = make(1, 4, 100, torch.float32)
    r = m.token_logprobs(x, t, top=2)
    g = torch.ones(4, device=DEV)
    for bad in (lambda: m.token_logprobs(x.double(), t), lambda: m.token_logprobs(x.half(), t),
                lambda: m.token_logprobs(x.t(), t[:1].expand(100)),
                lambda: m.token_logprobs(x[0], t), lambda: m.token_logprobs(x.cpu(), t),
                lambda: m.token_logprobs(x[:1].expand(4, 100), t),
                lambda: m.token_logprobs(x, t[:3]), lambda: m.token_logprobs(x, t.int()),
                lambda: m.token_logprobs(x, t, top=33), lambda: m.token_logprobs(x, t, top=-1),
                lambda: m.token_logprobs_backward(x, t, r.stats[:3], r.entropy, g),
                lambda: m.token_logprobs_backward(x, t, r.stats, r.entropy, g.double()),
                lambda: m.token_logprobs_backward(x, t, r.stats, r.entropy, g, top_id=r.top_id),
                lambda: m.token_logprobs_backward(x, t, r.stats, r.entropy, g, top_id=r.top_id,
                                                  grad_top=torch.ones(4, 3, device=DEV)),
                lambda: m.token_logprobs_backward(x, t, r.stats, r.entropy, g,
                                                  out=x[:3].clone()),
                lambda: m.token_logprobs_backward(x, t, r.stats, r.entropy, g,
                                                  out=x.bfloat16())):
        with pytest.raises(ValueError):
            bad()
    for temperature in (0.0, -1.0, float("nan"), INF, 1e-60):
        with pytest.raises(m.MXFP8Error) as e:
            m.token_logprobs(x, t, temperature)
        assert e.value.status == m.ERR_INVALID_ARG
    with pytest.raises(m.MXFP8Error):
        m.token_logprobs(x[:, :0], t)


@pytest.mark.parametrize("rows,vocab,dtype", [(2501, 517, torch.bfloat16), (2600, 130, torch.float32),
                                              (1300, 12500, torch.bfloat16),
                                              (1250, 6400, torch.float32)])
@pytest.mark.parametrize("top", [0, 7, 32])
def test_many_rows_of_smaller_vocabularies(m, rows, vocab, dtype, top):
    """Enough rows for CTAs of 64 and of 128 threads; some rows tied, masked or empty."""
    x, t = make(rows + top, rows, vocab, dtype, vocab + 3, 1)
    x[5] = 2.0
    x[6, 3:] = -INF
    x[7] = -INF
    x[8] = torch.arange(vocab, device=DEV).to(dtype)
    x[9, ::2] = torch.finfo(dtype).min
    x[10, 11] = float("nan")
    t[8:11] = 4
    check_forward(m, x, t, 0.9, top)
