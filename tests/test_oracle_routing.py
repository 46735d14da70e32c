"""The CPU oracles of routing and of the gated activation, pinned by hand-worked plans, by
adjoints and by central differences."""
import numpy as np

import oracle.routing_oracle as R
import oracle.swiglu_oracle as S


def test_plan_by_hand():
    ids = np.array([[2, 0], [0, -1], [2, 2]])
    offsets, row_of, entry_of = R.route(ids, 4, 128)
    assert offsets.tolist() == [0, 32, 32, 64, 128]      # expert 1 empty, the rest left over
    assert row_of.tolist() == [[32, 0], [1, -1], [33, 34]]
    assert entry_of[:3].tolist() == [1, 2, -1]
    assert entry_of[32:36].tolist() == [0, 4, 5, -1]
    assert (entry_of >= 0).sum() == 5
    offsets, row_of, entry_of = R.route(ids, 4, 32)      # two experts need 64
    assert offsets.tolist() == [0, 0, 0, 0, 32]
    assert (row_of == -1).all() and (entry_of == -1).all()


def test_rows_fit_any_choice():
    g = np.random.default_rng(0)
    for _ in range(200):
        t, k, e = int(g.integers(0, 40)), int(g.integers(1, 9)), int(g.integers(1, 20))
        ids = g.integers(-1, e, (t, k))
        offsets, row_of, _ = R.route(ids, e, R.rows_for(t, k, e))
        assert ((row_of >= 0) == (ids >= 0)).all()


def test_dispatch_and_combine_are_adjoint():
    g = np.random.default_rng(1)
    ids = g.integers(-1, 5, (17, 3))
    rows = R.rows_for(17, 3, 5)
    _, row_of, entry_of = R.route(ids, 5, rows)
    x, y = g.standard_normal((17, 4)), g.standard_normal((rows, 4))
    w = g.standard_normal((17, 3))
    out, _ = R.combine(y, row_of, w)
    np.testing.assert_allclose((out * x).sum(), (y * R.dispatch(x, row_of, rows, w)).sum(),
                               rtol=1e-12)
    dw, _ = R.combine_weights_grad(x, y, row_of)
    np.testing.assert_allclose((out * x).sum(), (dw * w).sum(), rtol=1e-12)   # linear in w
    assert (R.dispatch(x, row_of, rows, w)[entry_of < 0] == 0).all()


def test_gated_activation_gradient_by_differences():
    g = np.random.default_rng(2)
    a, u, dh = g.standard_normal(400) * 4, g.standard_normal(400), g.standard_normal(400)
    step = 1e-5
    dg, du = S.backward(a, u, dh)
    np.testing.assert_allclose(
        dg, dh * (S.forward(a + step, u) - S.forward(a - step, u)) / (2 * step), atol=1e-8)
    np.testing.assert_allclose(
        du, dh * (S.forward(a, u + step) - S.forward(a, u - step)) / (2 * step), atol=1e-8)
    assert S.forward(np.array([-800.0]), np.array([1.0]))[0] == 0
