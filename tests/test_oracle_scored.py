"""The scored-routing oracle against hand-worked values, invariants and finite differences."""

import numpy as np
import pytest

from oracle import scored as SC


def _cfg(**kw):
    c = dict(S=6, G=2, E=8, k=3, capacity_factor=0.0, n_expert_groups=0, topk_groups=0)
    c.update(kw)
    return c


def test_hand_worked_token():
    """Sigmoids 0.5, 0.75, 0.25, 0.9 (logits ln of the odds); the bias lifts the third over the
    second, and the weights come from the sigmoids alone."""
    s = np.array([0.5, 0.75, 0.25, 0.9])
    logits = np.log(s / (1 - s))[None, :]
    cfg = _cfg(S=1, G=1, E=4, k=2)
    sc = dict(score="sigmoid", group_top=1, renorm=1, scale=2.0)
    r = SC.route(logits, np.array([0.0, 0.0, 0.6, 0.0]), cfg, sc)
    assert r["expert_id"].tolist() == [[3, 2]]
    np.testing.assert_allclose(r["gate"], [[2 * 0.9 / 1.15, 2 * 0.25 / 1.15]], rtol=1e-12)
    np.testing.assert_allclose(r["aux_loss"], 4 * (0.9 + 0.25) / 2.4 / 2, rtol=1e-12)
    # groups {0, 1} and {2, 3}: the best pair wins with group_top 2, the best single with 1
    g2 = _cfg(S=1, G=1, E=4, k=2, n_expert_groups=2, topk_groups=1)
    assert SC.select(logits, None, g2, dict(sc, group_top=2)).tolist() == [[1, 0]]
    assert SC.select(logits, None, g2, sc).tolist() == [[3, 2]]


def test_ties_and_saturation():
    logits = np.array([[40.0, 50.0, 60.0, 0.0]])     # three sigmoids equal to 1 in fp64
    cfg = _cfg(S=1, G=1, E=4, k=3)
    sc = dict(score="sigmoid", group_top=1, renorm=1, scale=1.0)
    assert SC.select(logits, None, cfg, sc).tolist() == [[0, 1, 2]]
    low = SC.route(np.full((1, 4), -900.0), None, cfg, sc)
    np.testing.assert_allclose(low["gate"], 1 / 3, rtol=1e-12)


def test_non_finite_experts_come_last_with_weight_zero():
    logits = np.array([[np.nan, 1.0, np.inf, -np.inf], [np.nan] * 4])
    cfg = _cfg(S=2, G=1, E=4, k=3)
    sc = dict(score="sigmoid", group_top=1, renorm=1, scale=1.0)
    r = SC.route(logits, None, cfg, sc)
    assert r["expert_id"].tolist() == [[1, 0, 2], [0, 1, 2]]
    np.testing.assert_array_equal(r["gate"], [[1, 0, 0], [0, 0, 0]])


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [0, 1])
@pytest.mark.parametrize("cf", [0.0, 0.5])
def test_gradient_by_differences(kind, renorm, cf):
    """Central differences with step h of a smooth fp64 function: error O(h^2) + O(eps / h)."""
    rng = np.random.default_rng(5)
    cfg = _cfg(capacity_factor=cf, n_expert_groups=4, topk_groups=2)
    sc = dict(score=kind, group_top=2, renorm=renorm, scale=2.5)
    logits = rng.standard_normal((cfg["S"], cfg["E"]))
    dgate = rng.standard_normal((cfg["S"], cfg["k"]))
    r = SC.route(logits, 0.1 * rng.standard_normal(cfg["E"]), cfg, sc)
    if cf:
        assert (r["pos"] < 0).any()
    g = SC.logit_grad(logits, cfg, sc, r, dgate, 0.3, 0.2)
    h = 1e-5
    for t in range(cfg["S"]):
        for e in range(cfg["E"]):
            up, dn = logits.copy(), logits.copy()
            up[t, e] += h
            dn[t, e] -= h
            num = (SC.loss(up, cfg, sc, r, dgate, 0.3, 0.2) - SC.loss(dn, cfg, sc, r, dgate, 0.3, 0.2)) / (2 * h)
            assert abs(num - g[t, e]) < 1e-8
