"""Losses on packed logits, for the oracle.

TEST INFRASTRUCTURE ONLY (see the package docstring).

The definitions, in float64 and one row or sequence at a time: token
log-probabilities, the paired preference loss and the clipped policy loss with
a KL term, each with its gradient by the chain rule through logp (dlogp / dz =
1[v == y] - softmax).
"""
import numpy as np


def rows_in(cu, labels, rows):
    """Rows with a target: label >= 0 and inside the packed sequences."""
    t = np.arange(rows)
    return (np.asarray(labels) >= 0) & (t >= cu[0]) & (t < cu[-1])


def token_logprobs(z, labels, use=None):
    """(logp [rows], softmax [rows, vocab]); 0 and zeros where use is false
    (default: a negative label)."""
    z = np.asarray(z, dtype=np.float64)
    labels = np.asarray(labels)
    use = labels >= 0 if use is None else use
    logp, p = np.zeros(len(z)), np.zeros_like(z)
    with np.errstate(invalid="ignore", divide="ignore"):
        for t in np.nonzero(use)[0]:
            e = np.exp(z[t] - z[t].max())
            p[t] = e / e.sum()
            if labels[t] >= z.shape[1]:
                logp[t], p[t] = np.nan, np.nan
            else:
                logp[t] = z[t, labels[t]] - z[t].max() - np.log(e.sum())
    return logp, p


def token_logprobs_bwd(p, labels, w, use=None):
    """Gradient of the logits for dLoss / dlogp = w."""
    labels = np.asarray(labels)
    use = labels >= 0 if use is None else use
    d = np.zeros_like(p)
    for t in np.nonzero(use)[0]:
        if w[t] == 0:
            continue
        d[t] = -w[t] * p[t]
        if labels[t] < p.shape[1]:
            d[t, labels[t]] += w[t]
    return d


def preference(z, labels, cu, ref=None, beta=0.1, kind="sigmoid", smooth=0.0, mean=False):
    """dict(loss, seq_logp, rewards, logp, w, dlogits)."""
    use = rows_in(cu, labels, len(z))
    logp, p = token_logprobs(z, labels, use)
    ref = np.zeros(len(z)) if ref is None else np.asarray(ref, dtype=np.float64)
    n = len(cu) - 1
    seq_logp, lr, div = np.zeros(n), np.zeros(n), np.ones(n)
    for i in range(n):
        at = [t for t in range(cu[i], cu[i + 1]) if use[t]]
        div[i] = max(1, len(at)) if mean else 1
        seq_logp[i] = logp[at].sum() / div[i]
        lr[i] = (logp[at] - ref[at]).sum() / div[i]
    w, total = np.zeros(len(z)), 0.0
    sig = lambda v: 1 / (1 + np.exp(-v))  # noqa: E731
    for k in range(n // 2):
        h = lr[2 * k] - lr[2 * k + 1]
        if kind == "sigmoid":
            total += (1 - smooth) * np.logaddexp(0, -beta * h) + smooth * np.logaddexp(0, beta * h)
            dh = -beta * ((1 - smooth) * sig(-beta * h) - smooth * sig(beta * h))
        elif kind == "hinge":
            total += max(0.0, 1 - beta * h)
            dh = -beta if beta * h < 1 else 0.0
        else:
            total += (h - 1 / (2 * beta)) ** 2
            dh = 2 * (h - 1 / (2 * beta))
        for i, s in ((2 * k, 1.0), (2 * k + 1, -1.0)):
            for t in range(cu[i], cu[i + 1]):
                if use[t]:
                    w[t] = s * dh / (n // 2) / div[i]
    return {"loss": total / (n // 2), "seq_logp": seq_logp, "rewards": beta * lr, "logp": logp,
            "w": w, "dlogits": token_logprobs_bwd(p, labels, w, use)}


def policy(z, labels, cu, adv, old=None, ref=None, lo=0.2, hi=0.2, kl_coef=0.0,
           reduction="token", token_adv=False):
    """dict(loss, kl, clip_frac, logp, w, dlogits)."""
    use = rows_in(cu, labels, len(z))
    logp, p = token_logprobs(z, labels, use)
    n = len(cu) - 1
    at = [[t for t in range(cu[i], cu[i + 1]) if use[t]] for i in range(n)]
    total, filled = sum(map(len, at)), sum(1 for a in at if a)
    w, loss, kls, hits = np.zeros(len(z)), 0.0, 0.0, 0
    for i in range(n):
        for t in at[i]:
            share = 1 / total if reduction == "token" else 1 / len(at[i]) / filled
            A = float(adv[t] if token_adv else adv[i])
            r = np.exp(logp[t] - (logp[t] if old is None else float(old[t])))
            u, c = -A * r, -A * min(max(r, 1 - lo), 1 + hi)
            cut = c > u
            loss += share * (c if cut else u)
            dterm = 0.0 if cut else u
            if ref is not None:
                d = float(ref[t]) - logp[t]
                kl = np.expm1(d) - d
                kls += share * kl
                loss += share * kl_coef * kl
                dterm -= kl_coef * np.expm1(d)
            hits += cut
            w[t] = share * dterm
    return {"loss": loss, "kl": kls, "clip_frac": hits / max(1, total), "logp": logp, "w": w,
            "dlogits": token_logprobs_bwd(p, labels, w, use)}
