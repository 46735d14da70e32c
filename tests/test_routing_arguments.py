"""Arguments of the routing calls and of the activation that the C interface's types do not hold."""
import pytest
import torch

import __graft_entry__
import mxfp8_block_scaled_05_gb300 as m


@pytest.fixture(scope="module", autouse=True)
def lib():
    __graft_entry__.build()
    return m.lib()


@pytest.mark.parametrize("tokens,top_k,experts", [
    (4, 2, 2 ** 32 + 4), (4, 2, 2 ** 31), (4, 2, -2 ** 32 + 4), (4, 2 ** 32 + 2, 4),
    (4, -2 ** 32 + 2, 4), (2 ** 64 + 4, 2, 4), (-2 ** 64 + 4, 2, 4), (4, 2, 1025), (-1, 2, 4)])
def test_route_rows_refuses_what_has_no_segments(tokens, top_k, experts):
    """The low 32 or 64 bits of a number are not taken for it."""
    with pytest.raises(ValueError, match="num_experts"):
        m.route_rows(tokens, top_k, experts)


@pytest.mark.gpu
def test_calls_refuse_what_does_not_fit():
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    ids, x = z(4, 2, d=torch.int64), z(4, 64)
    for experts in (2 ** 32 + 8, -2 ** 32 + 8, 2 ** 31, 1025, 0, -1):
        with pytest.raises(ValueError, match="num_experts"):
            m.route(ids, experts)
        with pytest.raises(m.MXFP8Error):
            m.route(ids, experts, 256)
    wide = 2 ** 32 + 2
    with pytest.raises(m.MXFP8Error):
        m.route(torch.empty(0, wide, dtype=torch.int64, device="cuda"), 8)
    plan = m.route(ids, 8)
    none = plan._replace(row_of=torch.empty(0, wide, dtype=torch.int32, device="cuda"))
    for call in (lambda: m.dispatch(x[:0], none), lambda: m.quantize_dispatch(x[:0], none),
                 lambda: m.combine(z(plan.entry_of.numel(), 64), none)):
        with pytest.raises(ValueError, match="top_k"):
            call()
    for rule in (2 ** 32, 2 ** 32 + 1, -2 ** 32, 2):
        with pytest.raises(m.MXFP8Error):
            m.swiglu(x, rule=rule)
    assert m.device_status() == m.OK
