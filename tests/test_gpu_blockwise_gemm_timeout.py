"""A pipeline wait that runs out in each shape of the block-wise GEMM: with a limit far below
the time of a block's first copies, the kernel latches ERR_TIMEOUT, waits for what it has in
flight and returns, and the same call is right again with the default limit. The limit is the
library's own; nothing here faults or hangs a GPU."""
import pytest
import torch

from tests.oracle_helpers import gpu_ready

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def m():
    mod = gpu_ready()
    yield mod
    mod.set_wait_limit_ns(0)
    assert mod.device_status() == mod.OK


def operands(mm, n, k, wgrad, pow2):
    g = torch.Generator(device=DEV).manual_seed(mm + n + k)
    kb = -(-k // 128)

    def codes(r):
        q = torch.randint(0, 256, (r, k), generator=g, device=DEV, dtype=torch.uint8)
        return torch.where((q & 0x7F) == 0x7F, q & 0x80, q)

    def scale(*shape):
        s = torch.exp2(torch.randint(-9, 6, shape, generator=g, device=DEV).float())
        return s if pow2 else s * 1.25
    return codes(mm), scale(kb, mm), codes(n), scale(kb, n) if wgrad else scale(-(-n // 128), kb)


CASES = {  # rows, columns, reduction, weight gradient, FP32 result, power-of-two scales
    "swapped, split": (5, 2048, 4096, False, False, False),
    "swapped, whole": (37, 24576, 1024, False, False, False),
    "single, split": (300, 512, 4096, False, True, False),
    "single, whole": (300, 8192, 384, False, False, False),
    "single weight gradient, split": (300, 512, 4096, True, True, False),
    "single weight gradient, whole": (1000, 2048, 384, True, True, False),
    "pair": (4096, 4096, 4096, False, False, False),
    "pair weight gradient": (6144, 4096, 4096, True, True, False),
    "block-scaled pair": (6144, 4096, 4096, True, True, True),
}


@pytest.mark.parametrize("name", CASES)
def test_wait_runs_out(m, name):
    mm, n, k, wgrad, fp32, pow2 = CASES[name]
    a, sa, b, sb = operands(mm, n, k, wgrad, pow2)
    args = (a, sa, b, sb, m.WGRAD if wgrad else m.FPROP, m.OUT_FP32 if fp32 else m.OUT_BF16)
    want = m.blockwise_gemm(*args)
    assert m.device_status() == m.OK
    flush = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)   # the operands leave L2
    hit = False
    try:
        for _ in range(10):
            flush.zero_()
            m.set_wait_limit_ns(1)
            m.blockwise_gemm(*args)
            status = m.device_status()
            m.set_wait_limit_ns(0)
            assert status in (m.OK, m.ERR_TIMEOUT)
            hit = hit or status == m.ERR_TIMEOUT
            assert torch.equal(m.blockwise_gemm(*args), want)     # after a time-out too
    finally:
        m.set_wait_limit_ns(0)
    assert hit, "no wait ran out"
    assert m.device_status() == m.OK
