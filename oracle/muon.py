"""The orthogonalised update (Newton-Schulz steps on the momentum, as the Muon
optimiser takes it), in float64 numpy, step by step on the matrix itself."""
import numpy as np

COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def orthogonalize(u, steps=5, coefficients=COEFFICIENTS, eps=1e-7):
    x = np.asarray(u, dtype=np.float64)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    with np.errstate(all="ignore"):
        x = x / max(np.sqrt((x * x).sum()), eps)
        a, b, c = coefficients
        for _ in range(steps):
            g = x @ x.T
            x = a * x + (b * g + c * (g @ g)) @ x
    return x.T if tall else x


def factor(adjust, rows, cols):
    return {None: 1.0, "shape": max(1.0, rows / cols) ** 0.5,
            "rms": 0.2 * max(rows, cols) ** 0.5}[adjust]


def step(p, g, m, lr, momentum=0.95, nesterov=True, weight_decay=0.0, adjust="shape", steps=5,
         coefficients=COEFFICIENTS, eps=1e-7):
    """(new p, new m)."""
    p, g, m = (np.asarray(t, dtype=np.float64) for t in (p, g, m))
    m = momentum * m + (1 - momentum) * g
    u = momentum * m + (1 - momentum) * g if nesterov else m
    o = orthogonalize(u, steps, coefficients, eps)
    return p * (1 - lr * weight_decay) - lr * factor(adjust, *p.shape) * o, m
