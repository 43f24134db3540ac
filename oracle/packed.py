"""Weights in 4 bits (oracle): the tiles' bytes from codes and scales and back,
place by place, in fp64. The pages count the experts' weights' traffic and print
no format; this is the one that include/moe_route.h describes.
"""
from __future__ import annotations

import numpy as np

from .rows import decode16

INT, E2M1 = 1, 2
VALUES = {INT: np.arange(16.0) - 8,
          E2M1: np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6])}


def tiles(n: int, size: int) -> int:
    return -(-n // size)


def tile_bytes(group: int) -> int:
    return 1024 + 16 * (128 // group) * 2


def place(r: int, c: int, codes: int) -> tuple[int, int]:
    """(byte, shift) in its tile of the code of row r and column c."""
    j, g, i = c // 32, c % 32 // 8, c % 8
    bit = 8 * (i % 4) + 4 * (i // 4) if codes == INT else 4 * i
    return 16 * (16 * g + r) + 4 * j + bit // 8, bit % 8


def _places(codes):
    return np.array([[place(r, c, codes) for c in range(128)] for r in range(16)])


def pack(q: np.ndarray, scale_bits: np.ndarray, codes: int, group: int) -> np.ndarray:
    """One matrix: q [rows, cols] codes 0 .. 15, scales [rows, ceil(cols /
    group)] as 16-bit patterns; past the end codes of zero and scales of 0."""
    rows, cols = q.shape
    nt, kt, per = tiles(rows, 16), tiles(cols, 128), 128 // group
    full = np.full((nt * 16, kt * 128), 8 if codes == INT else 0, np.uint8)
    full[:rows, :cols] = q
    s = np.zeros((nt * 16, kt * per), np.uint16)
    s[:rows, :scale_bits.shape[1]] = scale_bits
    at = _places(codes)
    out = np.zeros((nt, kt, tile_bytes(group)), np.uint8)
    for t in range(nt):
        for k in range(kt):
            part = full[16 * t:16 * t + 16, 128 * k:128 * k + 128]
            np.bitwise_or.at(out[t, k], at[..., 0], (part << at[..., 1]).astype(np.uint8))
            out[t, k, 1024:] = np.ascontiguousarray(s[16 * t:16 * t + 16, per * k:per * k + per]).view(np.uint8).ravel()
    return out.ravel()


def unpack(b: np.ndarray, rows: int, cols: int, codes: int, group: int, act: int):
    """(codes [rows, cols], scale of each of them) of one matrix."""
    nt, kt, per = tiles(rows, 16), tiles(cols, 128), 128 // group
    b = b.reshape(nt, kt, tile_bytes(group))
    at = _places(codes)
    q = (b[:, :, at[..., 0]] >> at[..., 1].astype(np.uint8)) & 15
    q = q.transpose(0, 2, 1, 3).reshape(nt * 16, kt * 128)[:rows, :cols]
    s = np.ascontiguousarray(b[:, :, 1024:]).view(np.uint16).reshape(nt, kt, 16, per)
    s = decode16(s.transpose(0, 2, 1, 3).reshape(nt * 16, kt * per), act).astype(np.float64)
    return q, np.repeat(s, group, axis=1)[:rows, :cols]


def matrix(b: np.ndarray, rows: int, cols: int, codes: int, group: int, act: int):
    """(values, sizes of what a kernel sums for each product) of one matrix in
    fp64: integer codes are summed as 0 .. 15 with 8 taken off."""
    q, s = unpack(b, rows, cols, codes, group, act)
    v = VALUES[codes][q] * s
    return v, (q + 8.0) * np.abs(s) if codes == INT else np.abs(v)
