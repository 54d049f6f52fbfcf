"""Pins of the head oracle: scipy's log_softmax, central differences of the loss
for both gradients, and rows that take no part."""
import numpy as np
import pytest
from scipy.special import log_softmax

from oracle import head


def _inputs(seed, T=7, D=5, V=11):
    rng = np.random.default_rng(seed)
    h, W = rng.standard_normal((T, D)), rng.standard_normal((V, D))
    y = rng.integers(0, V, T)
    y[2 % T] = -100
    return h, W, y


def test_logprobs_against_scipy():
    h, W, y = _inputs(0)
    logp, p = head.logprobs(h, W, y)
    ref = log_softmax(h @ W.T, axis=1)
    on = y >= 0
    assert np.allclose(logp[on], ref[np.arange(7), y.clip(0)][on], rtol=0, atol=1e-13)
    assert np.allclose(p[on], np.exp(ref)[on], rtol=1e-12)
    assert logp[2] == 0 and not p[2].any()


@pytest.mark.parametrize("reduction", ["mean", "sum"])
def test_gradients_by_differences(reduction):
    h, W, y = _inputs(1)
    _, _, dh, dW = head.cross_entropy(h, W, y, reduction)
    f = lambda: head.cross_entropy(h, W, y, reduction)[0]  # noqa: E731
    for x, d in ((h, dh), (W, dW)):
        for i in np.ndindex(x.shape):
            old, e = x[i], 1e-5
            x[i] = old + e
            up = f()
            x[i] = old - e
            down = f()
            x[i] = old
            assert abs((up - down) / (2 * e) - d[i]) < 1e-9


def test_weighted_gradients_by_differences():
    h, W, y = _inputs(2)
    w = np.random.default_rng(3).standard_normal(7)
    w[4] = 0
    dh, dW = head.gradients(h, W, y, head.logprobs(h, W, y)[1], w)
    f = lambda: float(head.logprobs(h, W, y)[0] @ w)  # noqa: E731
    for x, d in ((h, dh), (W, dW)):
        for i in np.ndindex(x.shape):
            old, e = x[i], 1e-5
            x[i] = old + e
            up = f()
            x[i] = old - e
            down = f()
            x[i] = old
            assert abs((up - down) / (2 * e) - d[i]) < 1e-9
    assert not dh[2].any() and not dh[4].any()


def test_rows_without_target_and_labels_past_the_vocabulary():
    h, W, y = _inputs(4)
    h[2] = np.nan
    loss, logp, dh, dW = head.cross_entropy(h, W, y)
    assert np.isfinite(loss) and np.isfinite(dW).all() and not dh[2].any()
    y[0] = 11
    loss, logp, dh, dW = head.cross_entropy(h, W, y)
    assert np.isnan(loss) and np.isnan(logp[0]) and np.isnan(dh[0]).all() and np.isnan(dW).all()
    assert np.isfinite(dh[1:]).all() and np.isfinite(logp[1:]).all()
    assert head.cross_entropy(h, W, np.full(7, -1))[0] == 0


def test_a_nearly_certain_target():
    h, W, y = _inputs(5, T=1)
    y[:] = 3
    W[3] = 40 * h[0] / (h[0] @ h[0])
    _, logp, dh, _ = head.cross_entropy(h, W, y)
    z = W @ h[0]
    other = np.exp(np.delete(z, 3) - z[3])
    ref = (other[:, None] * (np.delete(W, 3, 0) - W[3])).sum(0) / (1 + other.sum())
    assert np.allclose(dh[0], ref, rtol=1e-12, atol=0)
