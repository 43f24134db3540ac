"""Helpers for the GPU tests of the layer around the routing: seeded inputs
and the bounds that the kernels' outputs are held to.

u = 2^-24 is half a step of fp32 (round to nearest), HALF[act] that of the
activation format, relative to the value; below the format's normal numbers
half a step is absolute (TINY16). An e4m3 number is off by at most half its
step. Sums of n fp32 terms in any order are off by at most n u times the sum
of the terms' magnitudes where each addition rounds to nearest, twice that
where a matrix instruction's additions truncate.
"""
from __future__ import annotations

import numpy as np
import torch

import oracle
from combine_router_topk_amd import binding as B
from oracle import layer as L
from pathcheck import bits_to_tensor, host, tensor_bits  # noqa: F401

U = 2.0 ** -24
HALF = {B.MOE_F16: 2.0 ** -11, B.MOE_BF16: 2.0 ** -8}
TINY16 = {B.MOE_F16: 2.0 ** -25, B.MOE_BF16: 2.0 ** -134}
ACTS = [B.MOE_F16, B.MOE_BF16]


def bits16(rng, shape, act, size=1.0):
    return oracle.encode16((rng.standard_normal(shape) * size).astype(np.float32), act)


def codes8(rng, shape):
    """e4m3 codes of normal values (no NaN)."""
    v = np.clip(rng.standard_normal(shape) * 110, -448, 448).astype(np.float32)
    return torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy().copy()


def scales(rng, shape, size=1.0):
    return ((rng.random(shape) + 0.5) * size).astype(np.float32)


def dev(a, act=None):
    """The array on the GPU: 16-bit patterns as the activation format, codes
    as e4m3."""
    if a is None:
        return None
    if a.dtype == np.uint16:
        return bits_to_tensor(a, act).cuda()
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t.view(torch.float8_e4m3fn) if a.dtype == np.uint8 else t


def codes_of(t):
    return t.detach().cpu().view(torch.uint8).numpy()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def assert_within(got, want, bound, what):
    bad = ~(np.abs(got - want) <= bound) & ~(np.isnan(got) & np.isnan(want))
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4], got[bad][:4], want[bad][:4],
                           np.broadcast_to(bound, got.shape)[bad][:4])


def round_bound(v, act):
    """Half a step of the activation format around v."""
    return HALF[act] * np.abs(v) + TINY16[act]


def check_rows8(codes, scale, v, dv, what):
    """8-bit rows against fp64 rows v that the kernel knows to within dv: the
    scale is its block's amax / 448 (one more rounding), and each value is v
    rounded to the codes' grid."""
    rows, cols = v.shape
    nb = L.blocks(cols)
    pad = lambda a: np.pad(a, ((0, 0), (0, nb * 128 - cols))).reshape(rows, nb, 128)  # noqa: E731
    amax, d = np.abs(pad(v)).max(axis=2), pad(dv).max(axis=2)
    want = np.maximum(amax, L.TINY) / 448
    assert_within(scale, want, d / 448 + 2 * U * want, what + " scale")
    s = L.spread(scale, cols)
    got = L.decode8(codes) * s
    # the grid's step where the kernel's v / s may lie, its quotient rounded once
    t = np.abs(v) / s * (1 + 2 * U) + dv / s
    assert_within(got, v, s * L.e4m3_step(np.minimum(t, 448)) / 2 * (1 + 4 * U) + dv + 4 * U * np.abs(v), what)
