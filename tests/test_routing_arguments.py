"""Arguments of the routing calls and of the activation that the C interface's types do not hold, and
the sizes that the binding works out by itself."""
import random

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


def sizes(n):
    g = random.Random(0)
    for _ in range(n):
        yield int(2 ** g.uniform(0, 22)), g.randint(1, 64), g.randint(1, 1024)


def test_rows_of_a_plan_are_the_librarys(lib):
    for tokens, top_k, experts in sizes(3000):
        want = lib.mxfp8_route_rows(tokens, top_k, experts)
        assert want and m._plan_rows(tokens * top_k, experts) == want
        assert m.route_rows(tokens, top_k, experts) == want
    assert m._plan_rows(0, 7) == m.route_rows(0, 3, 7) == lib.mxfp8_route_rows(0, 3, 7) == 0


def test_scales_of_a_copy_are_the_librarys(lib):
    for rows, k, experts in sizes(3000):
        for axis in (m.ROW, m.COL):
            want = lib.mxfp8_grouped_scale_bytes(32 * rows, 32 * k, experts, axis)
            assert want and m._copy_scale_bytes(32 * rows, 32 * k, experts, axis) == want
    # widths that only the column copy takes
    for rows, cols, experts in ((32, 8, 1), (96, 40, 3), (1024, 2056, 128)):
        assert m._copy_scale_bytes(rows, cols, experts, m.COL) == \
            lib.mxfp8_grouped_scale_bytes(rows, cols, experts, m.COL)
