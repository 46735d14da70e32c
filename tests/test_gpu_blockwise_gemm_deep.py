"""Long reductions of the block-wise GEMM whose products all have one sign, where an accumulator
that drops low bits drifts one way.

For every K up to 2^22 the sum is off by at most 2^-9 sum |a b|, and here sum |a b| = C_exact. A
BF16 result is rounded once after that; rounding is monotonic, so it lies between the roundings
of the two ends. (The 64-bit sums of the reference are exact to K 2^-53.)"""
import pytest
import torch

from tests.oracle_helpers import gpu_ready

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def m():
    mod = gpu_ready()
    yield mod
    assert mod.device_status() == mod.OK


def positive_operands(seed, mm, n, k):
    """Finite codes of positive sign, scales 1: a weight gradient's operands."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    kb = -(-k // 128)
    a, b = (torch.randint(1, 0x7F, (r, k), generator=g, device=DEV, dtype=torch.uint8)
            for r in (mm, n))
    return a, torch.ones(kb, mm, device=DEV), b, torch.ones(kb, n, device=DEV)


def sampled(a, b):
    """64-bit values of 8 rows and 16 columns, the first and the last among them."""
    ri = torch.linspace(0, a.shape[0] - 1, 8).long().to(DEV)
    ci = torch.linspace(0, b.shape[0] - 1, 16).long().to(DEV)
    ref = torch.zeros(8, 16, dtype=torch.double, device=DEV)
    for k0 in range(0, a.shape[1], 1 << 20):
        da, db = (q[i, k0:k0 + (1 << 20)].view(torch.float8_e4m3fn).double()
                  for q, i in ((a, ri), (b, ci)))
        ref += da @ db.t()
    return ri, ci, ref


@pytest.mark.parametrize("mm,n,k", [(1536, 2048, 32768 + 16), (2048, 2048, 1 << 18),
                                    (1024, 1024, 1 << 22)])
@pytest.mark.parametrize("fp32", [False, True])
def test_one_sign(m, mm, n, k, fp32):
    a, sa, b, sb = positive_operands(k, mm, n, k)
    ri, ci, ref = sampled(a, b)
    c = m.blockwise_gemm(a, sa, b, sb, m.WGRAD, m.OUT_FP32 if fp32 else m.OUT_BF16)
    got, off = c[ri][:, ci].double(), ref * 2.0 ** -9
    low, high = ((ref + s * off).to(torch.float64 if fp32 else torch.bfloat16).double()
                 for s in (-1, 1))
    assert ((low <= got) & (got <= high)).all(), ((got - ref).abs() / ref).max().item()


def test_fp32_results_of_power_of_two_scales_are_summed_in_chunks(m):
    """The tensor cores sum 512 products at a time, in 16 steps of 32 that each drop less than
    2^-23 of the sum, and FP32 registers add those sums, each rounding by 2^-24. A sum over all
    of K in the tensor cores would be off by some (K / 32) 2^-24 = 1.2e-4, twelve times the
    bound."""
    mm, n, k = 2048, 2048, 65536
    a, sa, b, sb = positive_operands(9, mm, n, k)
    ri, ci, ref = sampled(a, b)
    c = m.blockwise_gemm(a, sa, b, sb, m.WGRAD, m.OUT_FP32)
    folded = m.blockwise_gemm(a, sa, b, sb, m.WGRAD, m.OUT_FP32, scale_type=m.BW_FP32)
    assert not torch.equal(c, folded)               # it did run on the block-scaled MMA
    err = (c[ri][:, ci].double() - ref).abs()
    bound = ref * (16 * 2.0 ** -23 + k / 512 * 2.0 ** -24)
    assert (err <= bound).all(), (err / ref).max().item()
