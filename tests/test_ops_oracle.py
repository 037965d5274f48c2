"""The float64 references of the operators: gradients against central
differences, closed forms, and the empty cases."""
import numpy as np
import pytest

from oracle import ops


def directional(f, x, g, rng, h=1e-6):
    """<g, v> against (f(x + h v) - f(x - h v)) / 2 h along a random v.

    Truncation is h^2 / 6 times a third derivative of order 1, rounding
    eps |f| / h ~ 1e-9 relative for f of order 10: 1e-6 relative to the larger
    of |<g, v>| and the scale of f covers both."""
    v = rng.standard_normal(x.shape)
    want = (f(x + h * v) - f(x - h * v)) / (2 * h)
    got = float(np.sum(g * v))
    assert abs(got - want) <= 1e-6 * max(abs(want), 1.0), (got, want)


@pytest.mark.parametrize("temperature,kd,ce", [(1.0, 1.0, 0.0), (2.0, 0.7, 0.4), (0.5, 0.0, 1.0)])
def test_distill_gradient_is_the_difference(temperature, kd, ce):
    rng = np.random.default_rng(1)
    z = rng.standard_normal((4, 23)) * 2
    idx = np.array([[0, 5, 22], [3, 3, -1], [-1, 30, -1], [1, 2, 3]])   # repeated, padded, empty
    y = rng.standard_normal((4, 3))
    lab = np.array([5, -100, 7, 23])
    w = np.array([1.0, 0.5, 2.0, 0.0])
    kw = dict(labels=lab, temperature=temperature, kd=kd, ce=ce, weight=w)
    f = lambda x: ops.distill_loss(x, idx, y, **kw)[0].sum()  # noqa: E731
    losses, dz = ops.distill_loss(z, idx, y, **kw)
    directional(f, z, dz, rng)
    assert losses[3] == 0 and not dz[3].any()
    if ce == 0.0:
        assert losses[2] == 0 and not dz[2].any()


def test_distill_of_the_teacher_itself_is_zero():
    rng = np.random.default_rng(2)
    z = rng.standard_normal((2, 9))
    losses, dz = ops.distill_loss(z, np.tile(np.arange(9), (2, 1)), z + 3.0, temperature=1.5)
    assert np.abs(losses).max() < 1e-14 and np.abs(dz).max() < 1e-14


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [0, 4, 6])
def test_qk_gradients_are_the_differences(interleaved, rot):
    rng = np.random.default_rng(3)
    x, w, dy = rng.standard_normal((5, 3, 7)), rng.standard_normal(7), rng.standard_normal((5, 3, 7))
    rope = None
    if rot:
        ang = np.arange(11)[:, None] * 0.3 ** np.arange(rot // 2)
        rope = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    pos = np.array([0, 10, 3, -1, 7])
    kw = dict(positions=pos, rope=rope, eps=1e-3, interleaved=interleaved, offset=1.0)
    dx, dw = ops.qk_norm_rope_grad(dy, x, w, **kw)
    directional(lambda v: float(np.sum(dy * ops.qk_norm_rope(v, w, **kw))), x, dx, rng)
    directional(lambda v: float(np.sum(dy * ops.qk_norm_rope(x, v, **kw))), w, dw, rng)


def test_qk_norm_keeps_the_length_and_position_zero_turns_nothing():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((2, 2, 8))
    ang = np.arange(4)[:, None] * 0.5 ** np.arange(4)
    rope = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    y = ops.qk_norm_rope(x, None, np.array([0, 3]), rope, eps=0.0)
    np.testing.assert_allclose(np.sum(y * y, -1), 8.0, rtol=1e-12)
    np.testing.assert_allclose(y[0], x[0] / np.sqrt(np.mean(x[0] ** 2, -1, keepdims=True)), rtol=1e-12)


def test_embedding_gradient_is_the_difference():
    rng = np.random.default_rng(5)
    tok = np.array([2, 0, 2, -1, 9, 2])
    table, dout = rng.standard_normal((4, 3)), rng.standard_normal((6, 3))
    grad, _, count = ops.embedding_grad(dout, tok, 4, 1.5)
    directional(lambda t: float(np.sum(dout * ops.embedding(t, tok, 1.5))), table, grad, rng)
    assert count.tolist() == [1, 0, 3, 0] and not grad[1].any()
    order, slot, rows, index, u = ops.embedding_plan(tok, 4)
    assert order.tolist() == [1, 0, 2, 5, 3, 4] and slot.tolist() == [0, 1, 1, 1, -1, -1]
    assert rows.tolist() == [0, 2, -1, -1] and index.tolist() == [0, -1, 1, -1] and u == 2
