"""Pins of the oracle's losses: log-probabilities against scipy, hand-computed
values, invariants, and gradients against central differences."""
import numpy as np
import pytest
from scipy.special import log_softmax

from oracle import loss


def _case(seed, lens, V, lead=0, tail=0, drop=0.2):
    rng = np.random.default_rng(seed)
    cu = np.cumsum([lead] + lens)
    rows = int(cu[-1]) + tail
    z = rng.standard_normal((rows, V)) * 2
    labels = rng.integers(0, V, rows)
    labels[rng.random(rows) < drop] = -100
    return rng, z, labels, cu


def _difference(f, z, labels, use, count, rng):
    h = 1e-6
    for _ in range(count):
        t, v = rng.integers(len(z)), rng.integers(z.shape[1])
        if rng.random() < 0.4 and labels[t] >= 0:
            v = labels[t]
        zp, zm = z.copy(), z.copy()
        zp[t, v] += h
        zm[t, v] -= h
        yield t, v, (f(zp) - f(zm)) / (2 * h)


def test_logprobs_against_scipy():
    _, z, labels, _ = _case(0, [9], 17)
    logp, p = loss.token_logprobs(z, labels)
    ref = log_softmax(z, axis=1)
    for t, y in enumerate(labels):
        assert logp[t] == pytest.approx(ref[t, y] if y >= 0 else 0.0, abs=1e-13)
    assert np.allclose(p.sum(1), labels >= 0)


def test_logprobs_special_rows():
    z = np.array([[0.0, -np.inf, 0.0], [-np.inf] * 3, [np.inf, 0, 0], [1, 2, 3]])
    logp, _ = loss.token_logprobs(z, [0, 1, 0, 5])
    assert logp[0] == pytest.approx(-np.log(2)) and np.isnan(logp[1:]).all()


@pytest.mark.parametrize("kind,smooth,mean", [("sigmoid", 0.0, False), ("sigmoid", 0.2, True),
                                              ("hinge", 0.0, False), ("ipo", 0.0, True)])
def test_preference_gradient(kind, smooth, mean):
    rng, z, labels, cu = _case(1, [4, 3, 0, 5], 11, lead=1, tail=2)
    ref = rng.standard_normal(len(z)) - 2
    f = lambda x: loss.preference(x, labels, cu, ref, 0.3, kind, smooth, mean)["loss"]  # noqa: E731
    o = loss.preference(z, labels, cu, ref, 0.3, kind, smooth, mean)
    for t, v, d in _difference(f, z, labels, None, 60, rng):
        assert o["dlogits"][t, v] == pytest.approx(d, abs=2e-8)
    assert not o["dlogits"][0].any() and not o["dlogits"][-2:].any()


def test_preference_known_values():
    _, z, labels, cu = _case(2, [3, 3], 5, drop=0.0)
    same = loss.preference(z, labels, cu, loss.token_logprobs(z, labels)[0])
    assert same["loss"] == pytest.approx(np.log(2)) and np.allclose(same["rewards"], 0)
    empty = loss.preference(z, labels, [0, 0, 0])
    assert empty["loss"] == pytest.approx(np.log(2)) and not empty["dlogits"].any()


@pytest.mark.parametrize("reduction,kl,token_adv", [("token", 0.0, False), ("token", 0.1, True),
                                                    ("sequence", 0.1, False)])
def test_policy_gradient(reduction, kl, token_adv):
    rng, z, labels, cu = _case(3, [4, 0, 5, 3], 11, lead=2, tail=1)
    logp = loss.token_logprobs(z, labels)[0]
    old, ref = logp + 0.3 * rng.standard_normal(len(z)), logp + rng.standard_normal(len(z))
    adv = rng.standard_normal(len(z) if token_adv else 4)
    run = lambda x: loss.policy(x, labels, cu, adv, old, ref, 0.2, 0.3, kl, reduction,  # noqa: E731
                                token_adv)
    o = run(z)
    assert 0 < o["clip_frac"] < 1
    for t, v, d in _difference(lambda x: run(x)["loss"], z, labels, None, 60, rng):
        assert o["dlogits"][t, v] == pytest.approx(d, abs=2e-8)


def test_policy_known_values():
    _, z, labels, cu = _case(4, [3, 4], 5, drop=0.0)
    o = loss.policy(z, labels, cu, [1.0, -2.0])
    assert o["loss"] == pytest.approx((-3 + 8) / 7) and o["clip_frac"] == 0
    assert np.allclose(o["w"], np.array([-1] * 3 + [2] * 4) / 7)
    o = loss.policy(z, labels, cu, [1.0, -2.0], reduction="sequence")
    assert o["loss"] == pytest.approx((-1 + 2) / 2)
    none = loss.policy(z, [-1] * 7, cu, [1.0, -2.0])
    assert none["loss"] == 0 and not none["dlogits"].any()
