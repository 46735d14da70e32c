"""Power-of-two scales: the block-scaled MMA is taken where it is estimated to pay, and the
folding kernel elsewhere. Few tiles with a long reduction, which only the folding kernel can
split over CTAs, are folded (512 x 512 x 200000: 109 us, 391 on the block-scaled MMA).

Which one ran shows in the bits: the two sum in different orders. Error on the block-scaled
MMA: each step of 32 products drops less than 2^-23 of the sum, so (K / 32) 2^-23 sum |a b|
over all of K for BF16, and (512 / 32) 2^-23 sum |a b| plus an FP32 sum of K / 512 terms, each
step rounding by 2^-24, for FP32. A BF16 result is rounded once after that; rounding is
monotonic, so it lies between the roundings of the two ends."""
import pytest
import torch

from tests.oracle_helpers import gpu_ready
from tests.test_gpu_blockwise_gemm_pow2 import operands, sampled

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def m():
    mod = gpu_ready()
    yield mod
    assert mod.device_status() == mod.OK


def both(m, ops, wgrad, dtype):
    op = m.WGRAD if wgrad else m.FPROP
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    return m.blockwise_gemm(*ops, op, dtype), m.blockwise_gemm(*ops, op, dtype, workspace=none)


@pytest.mark.parametrize("mm,n,k", [(512, 512, 200000), (1024, 1024, 65536), (264, 200, 1 << 20)])
@pytest.mark.parametrize("wgrad", [False, True])
@pytest.mark.parametrize("fp32", [False, True])
def test_long_reductions_of_few_tiles_are_folded(m, mm, n, k, wgrad, fp32):
    dtype = m.OUT_FP32 if fp32 else m.OUT_BF16
    c, folded = both(m, operands(k, mm, n, k, wgrad), wgrad, dtype)
    assert torch.equal(c, folded)
    assert m.blockwise_gemm_workspace_bytes(mm, n, k, dtype) == 0


@pytest.mark.parametrize("mm,n,k,wgrad,fp32", [
    (4096, 4096, 4096, False, False), (1000, 4104, 4112, True, False),
    (2056, 2048, 8192, True, True), (4000, 6152, 4096, False, False),
    (400, 24584, 4096, True, True)])
def test_where_it_pays(m, mm, n, k, wgrad, fp32):
    ops = operands(mm + k, mm, n, k, wgrad)
    c, folded = both(m, ops, wgrad, m.OUT_FP32 if fp32 else m.OUT_BF16)
    assert not torch.equal(c, folded)
    ri, ci, ref, ab = sampled(*ops, wgrad, 5)
    off = ab * (16 * 2.0 ** -23 + k / 512 * 2.0 ** -24 if fp32 else k / 32 * 2.0 ** -23)
    got = c[ri][:, ci].double()
    low, high = ((ref + s * off).to(torch.float64 if fp32 else torch.bfloat16).double()
                 for s in (-1, 1))
    assert ((low <= got) & (got <= high)).all(), ((got - ref).abs() / off).max().item()
    other = tuple(o.clone() for o in ops)
    other[1].view(-1)[3] *= 1.5                 # not a power of two: folded
    c, folded = both(m, other, wgrad, m.OUT_FP32 if fp32 else m.OUT_BF16)
    assert torch.equal(c, folded)


@pytest.mark.parametrize("mm,n,k,wgrad,fp32", [(4096, 4096, 4096, False, False),
                                               (2056, 2048, 8192, True, True)])
def test_caller_states_the_scale_type(m, mm, n, k, wgrad, fp32):
    """BW_FP32 folds without a look at the scales (and without a workspace); BW_POW2 is the
    default's result."""
    ops = operands(mm, mm, n, k, wgrad)
    op, dtype = m.WGRAD if wgrad else m.FPROP, m.OUT_FP32 if fp32 else m.OUT_BF16
    c, folded = both(m, ops, wgrad, dtype)
    assert not torch.equal(c, folded)
    out = torch.empty_like(c)
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    m.blockwise_gemm(*ops, op, dtype, out=out, scale_type=m.BW_FP32)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
    assert torch.equal(out, folded)
    assert torch.equal(m.blockwise_gemm(*ops, op, dtype, scale_type=m.BW_POW2), c)
    with pytest.raises(ValueError):
        m.blockwise_gemm(*ops, op, dtype, scale_type=2)
