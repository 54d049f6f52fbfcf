"""The language-model head's log-probabilities and cross entropy from hidden
states, with their gradients, in float64 numpy.

z = h W^T; logp_t = z_ty - log sum_v exp z_tv (0 without target, NaN for a label
past the vocabulary); for weights w = dLoss / dlogp: dz = w (1[y] - p),
dh = dz W, dW = dz^T h.  Rows without target, or of weight 0, take no part.
"""
import numpy as np


def logprobs(h, W, labels):
    """(logp [T], p [T, V]) of float64 h [T, D] and W [V, D]."""
    labels = np.asarray(labels)
    T, V = h.shape[0], W.shape[0]
    logp, p = np.zeros(T), np.zeros((T, V))
    for t in np.nonzero(labels >= 0)[0]:
        if labels[t] >= V:
            logp[t], p[t] = np.nan, np.nan
            continue
        with np.errstate(all="ignore"):
            z = W @ h[t]
            m = z.max()
            e = np.exp(z - m)
            s = e.sum()
            p[t] = e / s
            logp[t] = z[labels[t]] - m - np.log(s)
    return logp, p


def gradients(h, W, labels, p, w):
    """(dh, dW) for dLoss / dlogp = w [T]."""
    labels, w = np.asarray(labels), np.asarray(w, dtype=np.float64)
    on = (labels >= 0) & (w != 0)
    dz = -w[on, None] * p[on]
    y = labels[on]
    inside = np.nonzero(y < W.shape[0])[0]
    # 1 - p of the target as the sum of the others
    rest = p[on][inside].copy()
    rest[np.arange(len(inside)), y[inside]] = 0
    dz[inside, y[inside]] = w[on][inside] * rest.sum(1)
    dh = np.zeros_like(h)
    dh[on] = dz @ W
    return dh, dz.T @ h[on]


def cross_entropy(h, W, labels, reduction="mean"):
    """(loss, logp, dh, dW)."""
    logp, p = logprobs(h, W, labels)
    n = int((np.asarray(labels) >= 0).sum())
    k = 1.0 / max(n, 1) if reduction == "mean" else 1.0
    dh, dW = gradients(h, W, labels, p, np.full(len(logp), -k))
    return -logp.sum() * k, logp, dh, dW
