"""The block-wise GEMM of power-of-two scales with a workspace: the block-scaled MMA runs if
every scale is a power of two, and the folding kernel if a single one is not.

The tensor cores then accumulate over all of K, each addition losing at most 2^-23 of the
running magnitude: |C - C_exact| <= K 2^-23 sum |a b|, and BF16 rounds once more. For an FP32
result they accumulate over 512 at a time, and FP32 registers add those sums up:
|C - C_exact| <= (512 2^-23 + (K / 512) 2^-24) sum |a b|."""
import pytest
import torch

from tests.oracle_helpers import gpu_ready

pytestmark = pytest.mark.gpu
DEV = "cuda"
SIZES = [(2048, 6152, 4112, False), (1021, 12288, 4096, False), (4104, 2056, 6144, True)]


@pytest.fixture(scope="module")
def m():
    mod = gpu_ready()
    yield mod
    assert mod.device_status() == mod.OK


def operands(seed, mm, n, k, wgrad):
    g = torch.Generator(device=DEV).manual_seed(seed)
    kb = -(-k // 128)

    def codes(r, c):
        q = torch.randint(0, 256, (r, c), generator=g, device=DEV, dtype=torch.uint8)
        return torch.where((q & 0x7F) == 0x7F, q & 0x80, q)

    def scale(*shape):
        return torch.exp2(torch.randint(-9, 6, shape, generator=g, device=DEV).float())
    return codes(mm, k), scale(kb, mm), codes(n, k), \
        scale(kb, n) if wgrad else scale(-(-n // 128), kb)


def sampled(a, sa, b, sb, wgrad, seed):
    """64-bit values of a sample of rows and columns, always the first and the last."""
    g = torch.Generator().manual_seed(seed)
    ri = torch.cat([torch.tensor([0, a.shape[0] - 1]), torch.randint(a.shape[0], (62,), generator=g)])
    ci = torch.cat([torch.tensor([0, b.shape[0] - 1]), torch.randint(b.shape[0], (126,), generator=g)])
    ri, ci = ri.to(DEV), ci.to(DEV)

    def deq(q, s):
        return q.view(torch.float8_e4m3fn).double() * \
            s.double().repeat_interleave(128, 1)[:, :q.shape[1]]
    da = deq(a[ri], sa[:, ri].t())
    db = deq(b[ci], sb[:, ci].t()) if wgrad else deq(b[ci], sb[ci // 128])
    return ri, ci, da @ db.t(), da.abs() @ db.abs().t()


@pytest.mark.parametrize("size", SIZES)
def test_power_of_two_scales(m, size):
    mm, n, k, wgrad = size
    ops = operands(mm, mm, n, k, wgrad)
    op = m.WGRAD if wgrad else m.FPROP
    assert m.blockwise_gemm_workspace_bytes(mm, n, k) > 0
    assert m.blockwise_gemm_workspace_bytes(mm, n, k, m.OUT_FP32) > 0
    c = m.blockwise_gemm(*ops, op)
    ri, ci, ref, ab = sampled(*ops, wgrad, 1)
    err = (c[ri][:, ci].double() - ref).abs()
    bound = ab * (k * 2.0 ** -23) + ref.abs() * 2.0 ** -8
    assert (err <= bound).all(), (err / bound).max().item()
    for _ in range(2):
        assert torch.equal(m.blockwise_gemm(*ops, op), c)


@pytest.mark.parametrize("size", SIZES + [(2056, 6152, 4400, True)])
def test_power_of_two_scales_fp32(m, size):
    mm, n, k, wgrad = size
    ops = operands(mm + 1, mm, n, k, wgrad)
    op = m.WGRAD if wgrad else m.FPROP
    out = torch.full((mm + 1, n), 7.0, device=DEV)
    c = m.blockwise_gemm(*ops, op, m.OUT_FP32, out=out[:mm])
    assert (out[mm] == 7.0).all()
    ri, ci, ref, ab = sampled(*ops, wgrad, 3)
    err = (c[ri][:, ci].double() - ref).abs()
    bound = ab * (512 * 2.0 ** -23 + k / 512 * 2.0 ** -24)
    assert (err <= bound).all(), (err / bound).max().item()
    for _ in range(2):
        assert torch.equal(m.blockwise_gemm(*ops, op, m.OUT_FP32), c)


@pytest.mark.parametrize("which,value", [("a", 3.0), ("b", 0.0)])
def test_one_other_scale_selects_the_folding_kernel_fp32(m, which, value):
    mm, n, k, _ = SIZES[2]
    a, sa, b, sb = operands(n, mm, n, k, True)
    (sa if which == "a" else sb).view(-1)[0] = value
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    plain = m.blockwise_gemm(a, sa, b, sb, m.WGRAD, m.OUT_FP32, workspace=none)
    assert torch.equal(m.blockwise_gemm(a, sa, b, sb, m.WGRAD, m.OUT_FP32), plain)


@pytest.mark.parametrize("size", SIZES[:1] + SIZES[2:])
@pytest.mark.parametrize("which,value", [("a", 3.0), ("b", 2.0 ** -20 * 1.0000001), ("a", -1.0),
                                         ("b", 0.0), ("a", 1e-42)])
def test_one_other_scale_selects_the_folding_kernel(m, size, which, value):
    mm, n, k, wgrad = size
    a, sa, b, sb = operands(n, mm, n, k, wgrad)
    s = sa if which == "a" else sb
    s.view(-1)[-1] = value
    op = m.WGRAD if wgrad else m.FPROP
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    plain = m.blockwise_gemm(a, sa, b, sb, op, workspace=none)
    assert torch.equal(m.blockwise_gemm(a, sa, b, sb, op), plain)


def test_extreme_powers_nan_and_given_workspace(m):
    mm, n, k, _ = SIZES[0]
    a, sa, b, sb = operands(7, mm, n, k, False)
    sa[0, 5], sb[:, 0] = 2.0 ** 100, 2.0 ** -127     # a subnormal power of two
    sa[3, 9], a[9, 384:512] = float("nan"), 0x7F
    ws = torch.full((m.blockwise_gemm_workspace_bytes(mm, n, k) + 64,), 0xAB, dtype=torch.uint8,
                    device=DEV)
    c = m.blockwise_gemm(a, sa, b, sb, workspace=ws)
    assert (ws[-64:] == 0xAB).all()
    assert c[9].isnan().all() and not c[8].isnan().any() and not c[10].isnan().any()
    ri, ci, ref, ab = sampled(a, sa, b, sb, False, 2)
    keep = ~ref.isnan()
    err = (c[ri][:, ci].double() - ref).abs()
    assert (err <= ab * (k * 2.0 ** -23) + ref.abs() * 2.0 ** -8)[keep].all()


def test_replay_in_a_graph_follows_the_scales(m):
    """One captured call; the scales change between replays from powers of two to others."""
    mm, n, k, _ = SIZES[0]
    a, sa, b, sb = operands(8, mm, n, k, False)
    m.blockwise_gemm(a, sa, b, sb)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = m.blockwise_gemm(a, sa, b, sb)
    for factor in (1.0, 1.5, 1.0):
        sa.mul_(factor)
        graph.replay()
        want = m.blockwise_gemm(a, sa, b, sb)
        assert torch.equal(c, want)


def test_workspace_refusals(m):
    a, sa, b, sb = operands(1, 256, 256, 256, False)
    with pytest.raises(ValueError):
        m.blockwise_gemm(a, sa, b, sb, workspace=torch.empty(64, device=DEV))
    buf = torch.empty(64, dtype=torch.uint8, device=DEV)
    mm, n, k, _ = SIZES[0]
    a, sa, b, sb = operands(1, mm, n, k, False)
    with pytest.raises(m.MXFP8Error) as e:
        m.blockwise_gemm(a, sa, b, sb, workspace=buf[8:])
    assert e.value.status == m.ERR_ALIGNMENT
    # too small: as without one
    none = m.blockwise_gemm(a, sa, b, sb, workspace=buf)
    sa.view(-1)[0] *= 1.5
    assert not torch.equal(none, m.blockwise_gemm(a, sa, b, sb))


def test_wait_limit_is_reported_and_the_next_call_works_fp32(m):
    mm, n, k, _ = SIZES[2]
    ops = operands(9, mm, n, k, True)
    c = m.blockwise_gemm(*ops, m.WGRAD, m.OUT_FP32)
    assert m.device_status() == m.OK
    m.set_wait_limit_ns(1)
    try:
        m.blockwise_gemm(*ops, m.WGRAD, m.OUT_FP32)
        torch.cuda.synchronize()
        assert m.device_status() in (m.ERR_TIMEOUT, m.OK)
    finally:
        m.set_wait_limit_ns(0)
    assert torch.equal(m.blockwise_gemm(*ops, m.WGRAD, m.OUT_FP32), c)
    assert m.device_status() == m.OK
