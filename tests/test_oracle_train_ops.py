"""Pins of the training-step operators' oracle: closed forms, and gradients against differences."""

import numpy as np
import pytest

from oracle import train_ops as ops


def _numeric(f, x, h=1e-6):
    """The gradient of the scalar f at x by central differences."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + h
        up = f(x)
        x[i] = keep - h
        g[i] = (up - f(x)) / (2 * h)
        x[i] = keep
    return g


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_adds_angles(interleaved):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 3, 4, 10))
    a, b = rng.standard_normal((2, 3, 1, 3)), rng.standard_normal((2, 3, 1, 3))
    y = ops.rotate(x, np.cos(a), np.sin(a), interleaved)
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-14)
    assert np.array_equal(y[..., 6:], x[..., 6:])
    both = ops.rotate(y, np.cos(b), np.sin(b), interleaved)
    assert np.allclose(both, ops.rotate(x, np.cos(a + b), np.sin(a + b), interleaved), atol=1e-14)
    i, j = (2, 3) if interleaved else (1, 4)   # the second pair
    assert np.allclose(y[..., i] + 1j * y[..., j], (x[..., i] + 1j * x[..., j]) * np.exp(1j * a[..., 1]), atol=1e-14)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_gradient_against_differences(interleaved):
    rng = np.random.default_rng(1)
    x, g, w = rng.standard_normal((2, 2, 2, 6)), rng.standard_normal((2, 2, 2, 6)), rng.standard_normal(6)
    a = rng.standard_normal((2, 2, 1, 2))
    c, s = np.cos(a), np.sin(a)
    dx, dw = ops.norm_rope_backward(x, g, w, c, s, 1e-3, interleaved)
    assert np.allclose(dx, _numeric(lambda v: np.sum(g * ops.norm_rope(v, w, c, s, 1e-3, interleaved)), x), atol=1e-8)
    assert np.allclose(dw, _numeric(lambda v: np.sum(g * ops.norm_rope(x, v, c, s, 1e-3, interleaved)), w), atol=1e-8)


def test_norm_gives_unit_mean_square():
    x = np.random.default_rng(2).standard_normal((1, 5, 3, 8)) * 7
    y = ops.norm_rope(x, np.ones(8), np.ones((1, 5, 1, 4)), np.zeros((1, 5, 1, 4)), 0.0, False)
    assert np.allclose(np.mean(y * y, -1), 1.0, rtol=1e-14)


def test_sort_by_hand():
    off, slot, row = ops.moe_sort(np.array([[2, 0], [0, -1], [2, 7]]), 3)
    assert off.tolist() == [0, 2, 2, 4]
    assert slot.tolist() == [1, 2, 0, 4, ~3, ~5]
    assert row.tolist() == [[2, 0], [1, ~4], [3, ~5]]


def test_combine_of_dispatch_scales_by_the_weights_kept():
    rng = np.random.default_rng(3)
    ids = rng.integers(-1, 5, (9, 3))
    x, w = rng.standard_normal((9, 4)), rng.standard_normal((9, 3))
    _, _, row = ops.moe_sort(ids, 5)
    kept = np.where(ids >= 0, w, 0.0).sum(1, keepdims=True)
    assert np.allclose(ops.moe_combine(ops.moe_dispatch(x, row), row, w), kept * x, atol=1e-14)


def test_moe_gradients_against_differences():
    rng = np.random.default_rng(4)
    ids = rng.integers(-1, 4, (5, 2))
    _, _, row = ops.moe_sort(ids, 4)
    y, w, g = rng.standard_normal((10, 3)), rng.standard_normal((5, 2)), rng.standard_normal((5, 3))
    dy, dw = ops.moe_combine_backward(g, y, row, w)
    assert np.allclose(dy, _numeric(lambda v: np.sum(g * ops.moe_combine(v, row, w)), y), atol=1e-8)
    assert np.allclose(dw, _numeric(lambda v: np.sum(g * ops.moe_combine(y, row, v)), w), atol=1e-8)
    x, gs = rng.standard_normal((5, 3)), rng.standard_normal((10, 3))
    assert np.allclose(ops.moe_combine(gs, row), _numeric(lambda v: np.sum(gs * ops.moe_dispatch(v, row)), x), atol=1e-8)


@pytest.mark.parametrize("rest", [False, True])
@pytest.mark.parametrize("ids", [[3, 0, 5], [3, -1, 5], [3, 5, 3], [-1, 9, -2]])
def test_distill_gradient_against_differences(ids, rest):
    rng = np.random.default_rng(5)
    z, t = rng.standard_normal(7), rng.standard_normal(3)
    lse = ops._lse(t / 1.7) + 0.4 if rest else None
    row = ops.distill_row(z, ids, t, 1.7, lse, 0.3)
    want = _numeric(lambda v: 0.3 * ops.distill_row(v, ids, t, 1.7, lse)["loss"], z)
    assert np.allclose(row["dlogits"], want, atol=1e-8)


def test_distill_of_the_student_itself_is_zero():
    rng = np.random.default_rng(6)
    z = rng.standard_normal(11)
    ids = rng.permutation(11)
    row = ops.distill_row(z, ids, z[ids], 2.0)   # all tokens, the same logits
    assert abs(row["loss"]) < 1e-14 and np.max(np.abs(row["dlogits"])) < 1e-15
    ids = ids[:4]                                # some tokens, and the mass of the others
    row = ops.distill_row(z, ids, z[ids], 2.0, ops._lse(z / 2.0))
    assert abs(row["loss"]) < 1e-14 and np.max(np.abs(row["dlogits"])) < 1e-15


def test_distill_rows_without_teacher():
    z = np.array([np.nan, 1.0, 2.0])
    for ids, t in (([-1, 3], [0.0, 0.0]), ([0, 1], [-np.inf, -np.inf])):
        row = ops.distill_row(z, ids, t, 1.0)
        assert row["loss"] == 0 and not row["dlogits"].any()
    z = np.zeros(3)
    assert ops.distill_row(z, [0, 1], [-np.inf, 0.0], 1.0)["loss"] == pytest.approx(np.log(3))
    assert ops.distill_row(np.array([-np.inf, 0.0]), [0], [0.0], 1.0)["loss"] == np.inf


@pytest.mark.parametrize("z_size,ids,lse_off", [
    (7, [3, 0, 5], -0.06),     # the pairs' p sum to more than 1: the teacher's logsumexp is too small
    (7, [3, 0, 5], -0.6),
    (7, [3, 5, 3], None),      # one token listed twice, the logsumexp over distinct tokens
    (4, [3, 0, 2, 1], 0.4),    # every token paired: no class for the rest, whatever the sum
    (3, [2, 0, 1, 1], -0.2),
])
def test_distill_gradient_where_the_pairs_mass_is_not_one(z_size, ids, lse_off):
    rng = np.random.default_rng(8)
    z, t = rng.standard_normal(z_size), rng.standard_normal(len(ids))
    if lse_off is None:
        t[2] = t[0]
        lse = ops._lse(t[:2] / 1.7) + 0.01
    else:
        lse = ops._lse(t / 1.7) + lse_off
    row = ops.distill_row(z, ids, t, 1.7, lse, 0.3)
    want = _numeric(lambda v: 0.3 * ops.distill_row(v, ids, t, 1.7, lse)["loss"], z)
    assert row["p_rest"] == 0 and abs(row["p"].sum() - 1) > 0.05
    assert np.allclose(row["dlogits"], want, atol=1e-8)
