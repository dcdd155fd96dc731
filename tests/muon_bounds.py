"""How far the Muon step's form on the Gram matrix may be off its definition."""

import numpy as np

# coefficients and counts of steps, ns[0]^(2 steps) up to 2^43
LARGEST = [((3.4445, -4.775, 2.0315), 12), ((1.875, -1.25, 0.375), 23), ((1.5, -0.5, 0.0), 32),
           ((-3.4445, 4.775, -2.0315), 12)]


def factors(s, ns, steps):
    """T's eigenvalue and its derivative for the eigenvalues s of S0."""
    t, dt = np.ones_like(s), np.zeros_like(s)
    ds = np.ones_like(s)
    for _ in range(steps):
        q = ns[0] + ns[1] * s + ns[2] * s * s
        dq = (ns[1] + 2 * ns[2] * s) * ds
        t, dt = t * q, dt * q + t * dq
        s, ds = s * q * q, ds * q * q + 2 * s * q * dq
    return t, dt


def steps_bound(u, ns, steps, chain, eps=1e-7):
    """Frobenius norm of what 64-bit rounding may change in X = T X0.

    A perturbation E of S0 changes T by D o E in S0's eigenvectors, D the divided
    differences of T's eigenvalue (its derivative on the diagonal), and X by
    that times the singular values: at most max |D_ij| sigma_j |E|.  With
    |X0| = 1, |E| is below `chain` 2^-53 from u u^T, `chain` the additions that a
    sum runs through, and below 8 r 2^-53 from the steps, whose own roundings,
    shrunk by what their remaining steps amplify less, sum up like a series of
    ns[0]^-2.  Rounding T itself costs steps r 2^-53 |T|.  Twice that holds the
    second order, while ns[0]^(2 steps) |E| is well below 1."""
    r = min(u.shape)
    x = u / (np.linalg.norm(u) + eps)
    sigma = np.linalg.svd(x, compute_uv=False)
    s = sigma * sigma
    t, dt = factors(s, ns, steps)
    gap = s[:, None] - s[None, :]
    near = np.abs(gap) <= 1e-3 * np.maximum(s[:, None], s[None, :])
    steep = np.maximum(np.abs(dt)[:, None], np.abs(dt)[None, :])
    with np.errstate(divide="ignore", invalid="ignore"):
        d = np.where(near, steep, np.abs((t[:, None] - t[None, :]) / gap))
    unit = 2.0 ** -53
    return 2 * unit * ((chain + 8 * r) * np.max(d * sigma[None, :]) + steps * r * np.abs(t).max())
