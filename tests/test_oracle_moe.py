"""Pins of the mixture-of-experts oracle: hand-worked picks and layers, closed forms."""

import numpy as np

from oracle import moe


def test_picks_ties_and_nan():
    l = np.array([[1.0, 3, 3, 2], [0, 0, 0, 0], [5, np.nan, 7, np.nan], [-np.inf, 1, -np.inf, 0]])
    ids, w = moe.route(l, 3, True)
    assert ids.tolist() == [[1, 2, 3], [0, 1, 2], [1, 3, 2], [1, 3, 0]]
    assert np.allclose(w[0], np.array([1, 1, np.exp(-1)]) / (2 + np.exp(-1))) and np.allclose(w[1], 1 / 3)
    assert np.isnan(w[2]).all() and np.allclose(w[3], [np.e / (1 + np.e), 1 / (1 + np.e), 0])
    assert np.allclose(moe.route(l, 3, False)[1][1], 0.25)


def test_hand_worked_layer():
    """One value in, one ffn value, two experts: everything by hand."""
    x = np.array([[2.0], [-1.0]])
    router = np.array([[0.0], [1.0]])
    gate_up = np.array([[[1.0], [3.0]], [[-1.0], [0.5]]])     # expert 0: gate 1, up 3; expert 1: gate -1, up 0.5
    down = np.array([[[2.0]], [[10.0]]])
    r = moe.layer(x, router, gate_up, down, 1)
    # token 0 (logits 0, 2): expert 1, gate -2, up 1; token 1 (logits 0, -1): expert 0, gate -1, up -3
    assert r["ids"].tolist() == [[1], [0]] and r["weights"].tolist() == [[1.0], [1.0]]
    assert np.allclose(r["out"], [[10 * -2 / (1 + np.exp(2))], [2 * (-1 / (1 + np.e)) * -3]])


def test_shares_add_up_and_empty_rows_are_zero():
    rng = np.random.default_rng(1)
    x, router = rng.standard_normal((5, 8)), rng.standard_normal((6, 8))
    gu, dn = rng.standard_normal((6, 8, 8)), rng.standard_normal((6, 8, 4))
    whole = moe.layer(x, router, gu, dn, 2, False)
    parts = [moe.layer(x, router, gu[a:b], dn[a:b], 2, False, first=a)["out"] for a, b in ((0, 1), (1, 4), (4, 6))]
    assert np.allclose(sum(parts), whole["out"])
    none = ~(whole["ids"] == 0).any(1)
    assert none.any() and not parts[0][none].any()


def test_all_experts_picked_is_the_dense_mixture():
    rng = np.random.default_rng(2)
    x, router = rng.standard_normal((3, 8)), rng.standard_normal((4, 8))
    gu, dn = rng.standard_normal((4, 12, 8)), rng.standard_normal((4, 8, 6))
    r = moe.layer(x, router, gu, dn, 4)
    p = np.exp(x @ router.T)
    p /= p.sum(1, keepdims=True)
    h = np.einsum("efd,td->tef", gu, x)
    y = np.einsum("edf,tef->ted", dn, h[..., :6] / (1 + np.exp(-h[..., :6])) * h[..., 6:])
    assert np.allclose(r["out"], np.einsum("te,ted->td", p, y))
