"""Helpers for the GPU tests of packed weights: seeded codes and scales as device
bytes, and the fp64 matrices they stand for, made when asked for."""
from __future__ import annotations

import numpy as np
import torch

import oracle
from combine_router_topk_amd import binding as B
from oracle import packed as O

FORMATS = [(O.INT, 128), (O.INT, 64), (O.INT, 32), (O.E2M1, 32), (O.E2M1, 64), (O.E2M1, 128)]


class Weights:
    """E packed matrices [rows, cols]; every code occurs, scales spread over a
    factor of three. Codes past a matrix's end are random, its scales there 1."""

    def __init__(self, rng, E, rows, cols, codes, group, scale_act, size=None):
        self.rows, self.cols, self.codes, self.group, self.scale_act = rows, cols, codes, group, scale_act
        self.format = B.make_packed_format(codes, group, scale_act)
        nt, kt, per = O.tiles(rows, 16), O.tiles(cols, 128), 128 // group
        b = rng.integers(0, 256, (E, nt, kt, O.tile_bytes(group)), dtype=np.uint8)
        s = (rng.random((E, nt, kt, 16 * per)) + 0.5) * (size or 0.4 / cols ** 0.5)
        b[..., 1024:] = oracle.encode16(s.astype(np.float32), scale_act).view(np.uint8)
        self.bytes = b.reshape(E, -1)
        self.dev = torch.from_numpy(self.bytes).cuda()
        self.made = {}
        assert self.bytes.size == B.moe_packed_weight_bytes(self.format, E, rows, cols)

    def both(self, e):
        """(values, sizes of what is summed) of expert e."""
        if e not in self.made:
            self.made[e] = O.matrix(self.bytes[e], self.rows, self.cols, self.codes, self.group, self.scale_act)
        return self.made[e]
