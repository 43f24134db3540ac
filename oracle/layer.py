"""The layer around the routing (oracle): the root-mean-square norm with its
residual and its gradient, 8-bit rows, the experts' products and the whole
layer, in fp64.

The pages name the experts' products (METRO AllGather vs AllToAll for MoE
decode, section "Add the expert-weight traffic term") and print no formulas;
those here are the usual definitions, stated in each function. 16-bit values
are uint16 bit patterns, e4m3 values uint8 codes.
"""
from __future__ import annotations

import numpy as np

from .rows import decode16, encode16

BLOCK = 128
TINY = 2.0 ** -100


def _e4m3_table() -> np.ndarray:
    """Value of each e4m3 code (OCP form): sign, 4 exponent bits with bias 7,
    3 mantissa bits; no infinities, all ones is NaN, exponent 0 is subnormal."""
    t = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = np.nan if c & 127 == 127 else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        t[c] = -v if c & 128 else v
    return t


E4M3 = _e4m3_table()


def decode8(codes: np.ndarray) -> np.ndarray:
    return E4M3[np.asarray(codes, np.uint8)]


def e4m3_step(t: np.ndarray) -> np.ndarray:
    """Spacing of e4m3 numbers around t."""
    a = np.maximum(np.abs(t), 2.0 ** -6)
    return 2.0 ** (np.floor(np.log2(a)) - 3)


def round_e4m3(t: np.ndarray) -> np.ndarray:
    """The nearest e4m3 number, ties to even, at most 448 in magnitude."""
    s = e4m3_step(t)
    return np.clip(np.round(t / s) * s, -448.0, 448.0)


def blocks(cols: int) -> int:
    return -(-cols // BLOCK)


def spread(scale: np.ndarray, cols: int) -> np.ndarray:
    """A row's block scales at each of its columns."""
    return np.repeat(np.asarray(scale, np.float64), BLOCK, axis=-1)[..., :cols]


def quantise(v: np.ndarray):
    """8-bit rows of fp64 rows: (e4m3 numbers, scales), scale = max(amax,
    2^-100) / 448; NaN scales for blocks that hold a non-finite value."""
    rows, cols = v.shape
    nb = blocks(cols)
    p = np.zeros((rows, nb * BLOCK))
    p[:, :cols] = v
    p = p.reshape(rows, nb, BLOCK)
    amax = np.abs(p).max(axis=2)
    scale = np.where(np.isfinite(amax), np.maximum(amax, TINY) / 448.0, np.nan)
    return round_e4m3(v / spread(scale, cols)), scale


def values8(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """The values that 8-bit rows stand for."""
    return decode8(codes) * spread(scale, codes.shape[-1])


def matrix8(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """The values of a weight matrix [rows, cols] with 128 x 128 scales."""
    rows = np.repeat(np.asarray(scale, np.float64), BLOCK, axis=0)[:codes.shape[0]]
    return decode8(codes) * spread(rows, codes.shape[1])


def rms_norm(x, residual, gamma, eps, act):
    """(h bits or None, rstd, v): h = round16(x + residual), rstd =
    1 / sqrt(mean h^2 + eps), v = h rstd gamma."""
    h = decode16(x, act).astype(np.float64)
    hb = None
    if residual is not None:
        hb = encode16(decode16(x, act) + decode16(residual, act), act)
        h = decode16(hb, act).astype(np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return hb, rstd, h * rstd[:, None] * decode16(gamma, act).astype(np.float64)


def rms_norm_backward(dy, dh, h, gamma, rstd, act):
    """(dx, dgamma) in fp64, from the kernel's own rstd: n = h rstd, u = dy
    gamma, dx = rstd (u - n mean(u n)) + dh, dgamma = sum_t dy n."""
    dy, h, g = (decode16(a, act).astype(np.float64) for a in (dy, h, gamma))
    r = np.asarray(rstd, np.float64)[:, None]
    n, u = h * r, dy * g
    dx = r * (u - n * (u * n).mean(axis=1, keepdims=True))
    if dh is not None:
        dx = dx + decode16(dh, act)
    return dx, (dy * n).sum(axis=0)


def segments(counts, offsets, rows):
    """(expert, its send rows) of every expert with rows."""
    for e, (c, o) in enumerate(zip(counts, offsets)):
        if c:
            yield e, np.arange(o, o + c)


def expert_gemm(a, a_scale, src, k, w, w_scale, counts, offsets, rows):
    """(y, |a| |w|) [rows, N] in fp64: y[r] = w[e] a[r'] over each expert's
    segment, r' = src[r] / k or r, and the sum of the products' magnitudes."""
    y = np.zeros((rows, w.shape[1]))
    mag = np.zeros_like(y)
    for e, r in segments(counts, offsets, rows):
        rr = r if src is None else np.asarray(src)[r] // k
        av, wv = values8(a[rr], a_scale[rr]), matrix8(w[e], w_scale[e])
        y[r], mag[r] = av @ wv.T, np.abs(av) @ np.abs(wv).T
    return y, mag


def silu(t):
    with np.errstate(over="ignore"):
        return t / (1.0 + np.exp(-t))


def moe_layer(x, idx, w, up, down, act):
    """(h bits [T, k, I], v, out): per pair v = silu(gate) * up of the token's
    row, h = round16(v), out = sum_j w down h; up [E, 2I, H] and down
    [E, H, I] are fp64 matrices."""
    T, k = idx.shape
    I = down.shape[2]
    xv = decode16(x, act).astype(np.float64)
    v = np.zeros((T, k, I))
    out = np.zeros((T, down.shape[1]))
    for t in range(T):
        for j in range(k):
            z = up[idx[t, j]] @ xv[t]
            v[t, j] = silu(z[:I]) * z[I:]
    h = encode16(v.astype(np.float32), act)
    hv = decode16(h, act).astype(np.float64)
    for t in range(T):
        for j in range(k):
            out[t] += float(w[t, j]) * (down[idx[t, j]] @ hv[t, j])
    return h, v, out
