"""Pins of the fp64 oracle of the operators around a block's products: closed forms, differences, brute force."""

import numpy as np
import pytest

from oracle import block_ops as ops


def test_norm_of_a_constant_row():
    x, y = np.full((1, 4), 3.0), np.full((1, 4), -2.0)
    r, h = ops.block_norm(x, y, None, None, None, True, 1.0, 0.5, 0.0)
    assert np.allclose(r, 2.5) and np.allclose(h, 1.0)          # y's norm is -1
    r, h = ops.block_norm(x, None, None, np.array([1.0, 2, 3, 4]), None, True, -1.0, 1.0, 0.0)
    assert np.allclose(r, -3.0) and np.allclose(h, [-1, -2, -3, -4])


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gates", [0, 1, 2, 6])
def test_block_gradients_by_differences(post, gates):
    rng = np.random.default_rng([gates, post])
    n, h = 6, 5
    v = {"x": rng.normal(size=(n, h)), "y": rng.normal(size=(n, h)), "w_pre": rng.normal(size=h)}
    if post:
        v["w_post"] = rng.normal(size=h)
    if gates:
        v["gate"] = rng.normal(size=(gates, h))
    g, dh = rng.normal(size=(n, h)), rng.normal(size=(n, h))

    def loss(v):
        r, out = ops.block_norm(v["x"], v["y"], v.get("w_post"), v["w_pre"], v.get("gate"), post, 0.7, 1.3, 1e-3)
        return np.sum(r * g) + np.sum(out * dh)

    got = ops.block_norm_backward(v["x"], v["y"], v.get("w_post"), v["w_pre"], v.get("gate"), post, 0.7, 1.3, 1e-3, g, dh)
    names = {"x": "dx", "y": "dy", "w_pre": "dw_pre", "w_post": "dw_post", "gate": "dgate"}
    for name, t in v.items():
        for at in np.ndindex(t.shape):
            up, down = {k: a.copy() for k, a in v.items()}, {k: a.copy() for k, a in v.items()}
            up[name][at] += 1e-6
            down[name][at] -= 1e-6
            assert abs((loss(up) - loss(down)) / 2e-6 - got[names[name]][at]) < 1e-6


def test_e4m3_grid_by_listing_it():
    grid = sorted({s * m * 2.0 ** e for s in (1, -1) for e in range(-9, 6) for m in range(16) if m * 2.0 ** e <= 448
                   and (m >= 8 or e == -9)})
    assert len(grid) == 253 and max(grid) == 448                # 2 x 126 finite magnitudes and zero
    assert np.array_equal(ops.e4m3(np.array(grid)), grid)
    for lo, hi in zip(grid, grid[1:]):
        mid = (lo + hi) / 2
        near = ops.e4m3(np.array([mid, mid + (hi - lo) / 64, mid - (hi - lo) / 64]))
        assert near[1] == hi and near[2] == lo and near[0] in (lo, hi)
        step = hi - lo
        assert (near[0] / step) % 2 == 0 or near[0] == 0        # ties to the even multiple
    assert np.isnan(ops.e4m3(np.nan))


@pytest.mark.parametrize("largest,e", [(448.0, 0), (448.0001, 1), (224.0, -1), (1.0, -8), (1.75, -8), (1.7500001, -7),
                                       (2.0 ** -140, -126), (3.4e38, 120)])
def test_exponent(largest, e):
    assert ops.exponent(largest) == e and ops.exponent(0.0) == 0


def test_quantize_a_block_and_groups():
    x = np.zeros((2, 130))
    x[0, :3], x[1, 129] = [896.0, -1.0, np.inf], 3.0
    q, s = ops.quantize(x, 1)
    assert s.tolist() == [[128, 127], [127, 120]] and q.shape == (2, 256)
    assert q[0, 0] == 448 and q[0, 1] == -0.5 and np.isnan(q[0, 2]) and q[1, 129] == 384
    q, s = ops.quantize(x, 128)
    assert s.tolist() == [[128, 120]]
    qt, st, written = ops.quantize_groups(np.ones((5, 2)), [0, 2, 2, 5])
    assert qt.shape == (2, 384) and written.tolist() == [True] * 256 + [False] * 128
    assert qt[0, 0] == 256 and qt[0, 2] == 0 and qt[0, 130] == 256 and qt[0, 131] == 0 and st[0, 0] == 127 - 8


def test_value_undoes_the_scales():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(200, 300))
    for tall in (1, 128):
        q, s = ops.quantize(x, tall)
        back = ops.value(q, s)[:, :300]
        top = np.abs(x).max()
        assert np.abs(back - x).max() <= top * 2.0 ** -4 and np.abs(q).max() <= 448


def test_clip_factor():
    assert ops.grad_norm([np.array([3.0]), np.array([4.0])]) == 5.0
    assert ops.clip_factor(5.0, 1.0, 0.0) == 0.2 and ops.clip_factor(0.5, 1.0, 0.0) == 1.0
    assert ops.clip_factor(0.0, 1.0, 0.0) == 1.0 and ops.clip_factor(np.inf, 1.0, 0.0) == 0.0
    assert np.isnan(ops.clip_factor(np.nan, 1.0, 0.0))
