"""The fp64 oracle of the operators around the layer, pinned to closed forms and central differences (CPU only)."""
import numpy as np
import pytest

from oracle import block_oracle as bo


def _diff(f, x, v, h):
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


def test_rmsnorm_closed_forms():
    y, rstd = bo.rmsnorm(np.array([[3.0, -4.0], [0.0, 0.0]]), np.array([1.0, 2.0]), 0.0 + 1e-30)
    np.testing.assert_allclose(y[0], [3 / np.sqrt(12.5), -8 / np.sqrt(12.5)], rtol=1e-14)
    assert np.all(y[1] == 0) and rstd[0] == pytest.approx(1 / np.sqrt(12.5))
    # scaling the input leaves the output
    h = np.random.default_rng(0).normal(size=(3, 7))
    np.testing.assert_allclose(bo.rmsnorm(5 * h, np.ones(7), 0.0)[0], bo.rmsnorm(h, np.ones(7), 0.0)[0], rtol=1e-13)


def test_rmsnorm_backward_matches_differences():
    rng = np.random.default_rng(1)
    h, w, dy, dh = rng.normal(size=(5, 9)), rng.normal(size=9), rng.normal(size=(5, 9)), rng.normal(size=(5, 9))
    eps = 1e-3
    rstd = bo.rmsnorm(h, w, eps)[1]
    gh, gw = bo.rmsnorm_backward(dy, h, w, rstd, dh)
    v, u = rng.normal(size=h.shape), rng.normal(size=w.shape)
    # second-order differences: error h^2 |f'''| / 6 plus 2^-53 / h
    assert np.sum(gh * v) == pytest.approx(
        _diff(lambda a: np.sum(dy * bo.rmsnorm(a, w, eps)[0]) + np.sum(dh * a), h, v, 1e-5), rel=1e-7, abs=1e-7)
    assert np.sum(gw * u) == pytest.approx(_diff(lambda a: np.sum(dy * bo.rmsnorm(h, a, eps)[0]), w, u, 1e-5),
                                           rel=1e-7, abs=1e-7)


def test_balanced_load_has_loss_one():
    T, E, K = 24, 6, 2
    ids = np.array([[(2 * t) % E, (2 * t + 1) % E] for t in range(T)])
    r = bo.balance_loss(np.zeros((T, E)), ids, 1.0, 0.0)
    assert r["loss"][1] == pytest.approx(1.0) and np.all(r["counts"] == T * K // E)
    assert r["loss"][2] == pytest.approx(np.log(E) ** 2)
    np.testing.assert_allclose(r["dlogits"], 0.0, atol=1e-17)
    # every token on one expert, with certainty: f = E / K on it, P = 1
    hot = np.full((T, E), -1e3)
    hot[:, 3] = 0.0
    r = bo.balance_loss(hot, np.full((T, 1), 3), 1.0, 0.0)
    assert r["loss"][1] == pytest.approx(E)


@pytest.mark.parametrize("cuts,masked", [(None, False), ([0, 4, 4, 11], True)])
def test_balance_gradient_matches_differences(cuts, masked):
    rng = np.random.default_rng(2)
    T, E, K = 11, 5, 2
    logits = rng.normal(size=(T, E))
    logits[2, 1] = -np.inf
    ids = np.argsort(-logits, axis=1)[:, :K]
    mask = rng.random(T) < 0.7 if masked else None
    r = bo.balance_loss(logits, ids, 0.3, 0.2, mask, cuts, dloss=1.7)
    v = rng.normal(size=logits.shape)
    f = lambda a: 1.7 * bo.balance_loss(a, ids, 0.3, 0.2, mask, cuts)["loss"][0]
    assert np.sum(r["dlogits"] * v) == pytest.approx(_diff(f, logits, v, 1e-5), rel=1e-7, abs=1e-9)
    if masked:
        assert not r["dlogits"][~mask].any() and r["counts"].sum() == K * mask.sum() and not r["counts"][1].any()


def test_empty_and_masked_out():
    r = bo.balance_loss(np.zeros((0, 4)), np.zeros((0, 2), dtype=int), 1.0, 1.0)
    assert not r["loss"].any() and not r["counts"].any()
    r = bo.balance_loss(np.ones((3, 4)), np.zeros((3, 2), dtype=int), 1.0, 1.0, mask=np.zeros(3))
    assert not r["loss"].any() and not r["dlogits"].any()
    dead = np.full((2, 4), -np.inf)
    r = bo.balance_loss(dead, np.zeros((2, 1), dtype=int), 1.0, 1.0)
    assert r["counts"][0, 0] == 2 and not r["probs"].any() and not r["dlogits"].any()


def test_router_backward_matches_differences():
    rng = np.random.default_rng(3)
    X, W, dl = rng.normal(size=(6, 4)), rng.normal(size=(4, 3)), rng.normal(size=(6, 3))
    dX, dW = bo.router_backward(dl, X, W)
    v, u = rng.normal(size=X.shape), rng.normal(size=W.shape)
    assert np.sum(dX * v) == pytest.approx(_diff(lambda a: np.sum(dl * (a @ W)), X, v, 1e-4), rel=1e-8)
    assert np.sum(dW * u) == pytest.approx(_diff(lambda a: np.sum(dl * (X @ a)), W, u, 1e-4), rel=1e-8)
    a, b = bo.router_backward(dl, X, W, np.ones_like(X), 2 * np.ones_like(W))
    np.testing.assert_allclose(a, dX + 1)
    np.testing.assert_allclose(b, dW + 2)
