"""Momentum and orthogonalisation by Newton-Schulz products (oracle, test infrastructure).

Source: the Muon optimiser as its author describes it (momentum, optionally
Nesterov's; five steps of the quintic X <- a X + (b A + c A A) X with A = X X^T
on the update divided by its Frobenius norm; a, b, c = 3.4445, -4.7750, 2.0315).

Readings taken:
  * the momentum's two operations are rounded to float32 each, as the other
    memories here; everything after it is in float64;
  * the norm has no added constant: a matrix of zeros stays zero;
  * a matrix with an entry that is not finite becomes NaN.
"""
from __future__ import annotations

import numpy as np

COEFS = (3.4445, -4.7750, 2.0315)


def newton_schulz(u: np.ndarray, steps: int = 5, coefs=None) -> np.ndarray:
    """`steps` steps on u / |u|_F in float64; coefs: None, one triple, or one for each step (float32 values)."""
    x = np.asarray(u, np.float64)
    norm = np.sqrt(np.sum(x * x))
    if not np.isfinite(norm):
        return np.full(x.shape, np.nan)
    if norm == 0:
        return x
    x = x / norm
    c = np.broadcast_to(np.asarray(COEFS if coefs is None else coefs, np.float32).astype(np.float64), (steps, 3))
    for a, b, d in c:
        g = x @ x.T if x.shape[0] <= x.shape[1] else x.T @ x
        p = b * g + d * (g @ g)
        x = a * x + (p @ x if x.shape[0] <= x.shape[1] else x @ p)
    return x


def muon_step(grad: np.ndarray, mem, beta: float, nesterov: bool, steps: int = 5, coefs=None, scale: float = 1.0) -> dict:
    """One step: {"mem", "u", "out"}; grad float32 or uint16 bf16 bits, mem float32 or None."""
    if grad.dtype == np.uint16:
        grad = (grad.astype(np.uint32) << 16).view(np.float32)
    b = np.float32(beta)
    with np.errstate(all="ignore"):
        if mem is None:
            u = grad
        else:
            mem = b * mem + grad
            u = grad + b * mem if nesterov else mem
    return {"mem": mem, "u": u, "out": scale * newton_schulz(u, steps, coefs)}
