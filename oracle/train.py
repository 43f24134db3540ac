"""What trains the experts' weights (oracle), in fp64: an AdamW step with states
as they are or as 8-bit rows, and the weights' gradient over the routed rows.

The pages train experts and print no formulas; those here are the usual
definitions, stated in each function.
"""
from __future__ import annotations

import numpy as np

from .layer import blocks, decode8, segments, spread


def adamw(w, g, m, v, lr, beta1, beta2, eps, decay, step, scale=1.0):
    """(w, m, v, size of the update's terms) after one step: m = b1 m + (1 - b1)
    g, v = b2 v + (1 - b2) g^2, w = w - lr decay w - lr (m / c1) / (sqrt(v / c2) +
    eps), ci = 1 - bi^step. The size is that of the update with the magnitudes of
    m's two terms in m's place."""
    w, g, m, v = (np.asarray(a, np.float64) for a in (w, g, m, v))
    g = g * scale
    mag = beta1 * np.abs(m) + (1 - beta1) * np.abs(g)
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    c1, c2 = 1 - beta1 ** step, 1 - beta2 ** step
    den = np.sqrt(v / c2) + eps
    with np.errstate(divide="ignore", invalid="ignore"):
        return w - lr * decay * w - lr * (m / c1) / den, m, v, abs(lr) * (mag / c1) / den


def state8(codes, scale):
    """The values of a flat 8-bit state."""
    return decode8(codes) * spread(scale, np.asarray(codes).shape[0])


def weight_grad(dy, a, src, k, counts, offsets, E):
    """(dW [E, N, K], |dy|^T |a|) in fp64: dW[e] = sum over the rows r of e's
    segment of dy[r]^T a[r'], r' = src[r] / k or r; values, not bits."""
    dw = np.zeros((E, dy.shape[1], a.shape[1]))
    mag = np.zeros_like(dw)
    for e, r in segments(counts, offsets, dy.shape[0]):
        rr = r if src is None else np.asarray(src)[r] // k
        dw[e], mag[e] = dy[r].T @ a[rr], np.abs(dy[r]).T @ np.abs(a[rr])
    return dw, mag


__all__ = ["adamw", "state8", "weight_grad", "blocks"]
