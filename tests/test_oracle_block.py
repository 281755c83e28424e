"""The fp64 reference of the operators around the expert layer, pinned on the
CPU: gradients against central differences, the norm and routing against direct
statements of their definitions."""
import math

import numpy as np
import pytest

from oracle import block as ob


def test_layer_norm_rows_are_normalized():
    x = np.random.default_rng(0).normal(3.0, 2.0, (5, 33))
    y, mean, rstd = ob.layer_norm_fwd(x, eps=0.0)
    assert np.allclose(y.mean(1), 0, atol=1e-14) and np.allclose((y ** 2).mean(1), 1)
    assert np.allclose(mean, x.mean(1)) and np.allclose(rstd, 1 / x.std(1))
    y, _, rstd = ob.layer_norm_fwd(np.full((1, 7), 2.5), np.ones(7), np.arange(7.0), eps=1e-4)
    assert np.allclose(y, np.arange(7.0)) and np.allclose(rstd, 100)


def test_layer_norm_gradients_against_differences():
    rng = np.random.default_rng(1)
    x, w, b, dy = rng.normal(size=(4, 9)), rng.normal(size=9), rng.normal(size=9), rng.normal(size=(4, 9))
    _, mean, rstd = ob.layer_norm_fwd(x, w, b)
    dx, dw, db = ob.layer_norm_bwd(dy, x, w, mean, rstd)
    loss = lambda x, w, b: float((ob.layer_norm_fwd(x, w, b)[0] * dy).sum())
    h = 1e-6
    for at in np.ndindex(x.shape):
        d = np.zeros_like(x)
        d[at] = h
        assert abs((loss(x + d, w, b) - loss(x - d, w, b)) / (2 * h) - dx[at]) < 1e-7
    for i in range(9):
        d = np.zeros(9)
        d[i] = h
        assert abs((loss(x, w + d, b) - loss(x, w - d, b)) / (2 * h) - dw[i]) < 1e-7
        assert abs((loss(x, w, b + d) - loss(x, w, b - d)) / (2 * h) - db[i]) < 1e-7


def test_grad_norm_and_factor():
    assert ob.grad_norm([np.array([3.0]), np.zeros((0,)), np.array([[0.0, -4.0]])]) == 5.0
    assert ob.grad_norm([np.array([3.0]), np.array([[0.0, -4.0]])], math.inf) == 4.0
    assert ob.grad_norm([]) == 0.0 and ob.grad_norm([], math.inf) == 0.0
    assert ob.clip_factor(5.0, 10.0) == 1.0 and ob.clip_factor(5.0, 1.0) == 1.0 / (5.0 + 1e-6)


def test_route_ties_masks_and_nan():
    inf = math.inf
    ids, w = ob.route([[1.0, 2.0, 2.0, 0.0], [-inf, -inf, 5.0, -inf], [-inf] * 4, [0.0, math.nan, inf, 1.0]], 2)
    assert ids.tolist() == [[1, 2], [2, -1], [-1, -1], [1, 2]]
    assert w[:3].tolist() == [[0.5, 0.5], [1.0, 0.0], [0.0, 0.0]] and np.isnan(w[3]).all()
    _, w = ob.route([[0.0, math.log(2.0), 0.0, -inf]], 1, renormalize=False)
    assert np.allclose(w, 0.5)


@pytest.mark.parametrize("renormalize", [True, False])
def test_moe_layer_is_the_weighted_sum(renormalize):
    rng = np.random.default_rng(2)
    E, H, inner, T, k = 5, 6, 4, 3, 2
    x, lg = rng.normal(size=(T, H)), rng.normal(size=(T, E))
    w13, w2 = rng.normal(size=(E, 2 * inner, H)), rng.normal(size=(E, H, inner))
    y, ids, p, bound = ob.moe_layer(x, lg, w13, w2, k, renormalize)
    for t in range(T):
        want = np.zeros(H)
        soft = np.exp(lg[t]) / np.exp(lg[t]).sum()
        top = np.argsort(-lg[t])[:k]
        for e in top:
            g = w13[e, :inner] @ x[t]
            want += soft[e] / (soft[top].sum() if renormalize else 1) * (w2[e] @ (g / (1 + np.exp(-g)) * (w13[e, inner:] @ x[t])))
        assert np.allclose(y[t], want) and set(ids[t]) == set(top.tolist())
    assert (bound > 0).all() and (bound < 1e-1 * np.abs(y).max() + 1).all()
