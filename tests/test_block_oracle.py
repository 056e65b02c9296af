"""The oracle of the operators round the routed layer, against hand values, closed forms and differences (no GPU)."""
import math

import numpy as np
import pytest

from oracle import block_oracle as bo


def test_norms_by_hand():
    y, r = bo.norm([[3.0, 4.0]], np.ones(2), eps=0.0)
    assert np.allclose(y, [[3 / math.sqrt(12.5), 4 / math.sqrt(12.5)]]) and np.allclose(r, 1 / math.sqrt(12.5))
    y, _ = bo.norm([[1.0, 3.0]], np.array([1.0, 2.0]), np.array([0.5, 0.0]), "layer", 0.0, 1.0)
    assert np.allclose(y, [[-2 + 0.5, 3.0]])
    h, m = bo.residual(np.array([[2.0, -4.0]]), np.array([[1.0, 1.0]]), np.float32([0.5]), 3.0, 2.0)
    assert np.allclose(h, [[5.0, -4.0]]) and np.allclose(m, [[5.0, 8.0]])
    h, _ = bo.residual(np.array([[2.0, -4.0]]), None, np.float16([1, 2]))
    assert np.allclose(h, [[2.0, -8.0]])


def test_activations():
    v = np.array([-100.0, -1.0, 0.0, 1.0, 100.0])
    assert np.allclose(bo.act("silu", v), [0, -1 / (1 + math.e), 0, 1 / (1 + math.exp(-1)), 100])
    assert np.allclose(bo.act("relu", v), [0, 0, 0, 1, 100])
    assert np.allclose(bo.act("gelu", v), [0, -0.15865525, 0, 0.84134475, 100])
    assert np.allclose(bo.act("gelu_tanh", v), [0, -0.15880801, 0, 0.84119199, 100])
    assert np.allclose(bo.act("sigmoid", v), [0, 1 / (1 + math.e), 0.5, math.e / (1 + math.e), 1])


def test_balance_by_hand():
    # Two tokens, two experts, p = (3/4, 1/4) and (1/2, 1/2); picks 0 and 0: f = (2, 0), P = (5/8, 3/8).
    l = np.log(np.array([[3.0, 1.0], [1.0, 1.0]]))
    c, n, mean, loss = bo.balance(l, np.array([[0], [0]]), None, 1, coef=0.5)
    assert c.tolist() == [[2, 0]] and n.tolist() == [2]
    assert np.allclose(mean, [[5 / 8, 3 / 8]]) and math.isclose(loss, 0.5 * 2 * 5 / 8)
    # A perfectly even router has loss coef, whatever the sequences.
    l = np.zeros((6, 3))
    ids = np.arange(6)[:, None] % 3
    assert math.isclose(bo.balance(l, ids, [0, 3, 3, 6], 1, "sigmoid")[3], 1.0)
    # Bad tokens and picks of nobody count for nothing.
    l[1] = -np.inf
    l[4, 0] = np.nan
    ids[1], ids[4] = -1, 7
    c, n, _, _ = bo.balance(l, ids, [0, 3, 3, 6], 1)
    assert c.tolist() == [[1, 0, 1], [0, 0, 0], [1, 0, 1]] and n.tolist() == [2, 0, 2]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_against_differences(score):
    rng = np.random.default_rng(3)
    T, E, k, off = 7, 5, 2, [0, 3, 3, 6]
    l = rng.normal(size=(T, E)) * 2
    l[1, 2] = -np.inf
    l[2] = -np.inf
    ids = rng.integers(0, E, (T, k))
    c, n, _, _ = bo.balance(l, ids, off, k, score, 0.3)
    d, m, inside = bo.balance_grad(l, off, k, c, n, score, 0.3, 2.0)
    assert inside.tolist() == [True] * 6 + [False] and (d[6] == 0).all() and (d[2] == 0).all()
    assert (np.abs(d) <= m + 1e-15).all()
    for t in range(T):
        for e in range(E):
            if np.isfinite(l[t, e]):
                up, dn = l.copy(), l.copy()
                up[t, e] += 1e-5
                dn[t, e] -= 1e-5
                num = (bo.balance(up, ids, off, k, score, 0.3)[3] - bo.balance(dn, ids, off, k, score, 0.3)[3]) / 2e-5
                assert abs(2.0 * num - d[t, e]) < 1e-9, (t, e)
