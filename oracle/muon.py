"""The Muon step (momentum, Newton-Schulz steps, decoupled decay) in fp64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).
"""

import numpy as np

COEFFICIENTS, STEPS = (3.4445, -4.775, 2.0315), 5


def orthogonalised(u, eps=1e-7, ns=COEFFICIENTS, steps=STEPS):
    """The update u [rows, cols] after `steps` Newton-Schulz steps."""
    x = np.asarray(u, np.float64)
    tall = x.shape[0] > x.shape[1]
    x = (x.T if tall else x) / (np.sqrt(np.sum(x * x)) + eps)
    for _ in range(steps):
        s = x @ x.T
        x = ns[0] * x + (ns[1] * s + ns[2] * (s @ s)) @ x
    return x.T if tall else x


def factor(adjust, rows, cols):
    if adjust == "original":
        return np.sqrt(max(1.0, rows / cols))
    return 0.2 * np.sqrt(max(rows, cols))


def step(p, g, m, lr, momentum, nesterov, weight_decay, eps=1e-7, adjust="original",
         ns=COEFFICIENTS, steps=STEPS):
    """(p, m) after one step; the hyperparameters are fp32 numbers."""
    f = lambda a: np.float64(np.float32(a))
    lr, mu, wd = f(lr), f(momentum), f(weight_decay)
    m = mu * np.asarray(m, np.float64) + (1 - mu) * np.asarray(g, np.float64)
    u = mu * m + (1 - mu) * np.asarray(g, np.float64) if nesterov else m
    x = orthogonalised(u, f(eps), ns, steps)
    return np.asarray(p, np.float64) * (1 - lr * wd) - lr * factor(adjust, *x.shape) * x, m
