"""Newton-Schulz orthogonalisation from its definition in 64 bits (numpy)."""
import numpy as np


def momentum_step(g, m, mu, nesterov):
    """(u, the new momentum)."""
    m = mu * m.astype(np.float64) + g.astype(np.float64)
    return (g.astype(np.float64) + mu * m if nesterov else m), m


def orthogonalize(u, steps, coeffs, eps, scale=1.0):
    """One matrix; coeffs: one (a, b, c) per step."""
    x = u.astype(np.float64)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    x = x / (np.sqrt((x * x).sum()) + eps)
    for k in range(steps):
        a, b, c = coeffs[k]
        gram = x @ x.T
        x = a * x + (b * gram + c * gram @ gram) @ x
    return scale * (x.T if tall else x)
