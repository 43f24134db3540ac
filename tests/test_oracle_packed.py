"""The packed weights' oracle and the package's packing, without a GPU."""
import numpy as np
import pytest
import torch

import oracle
from combine_router_topk_amd import binding as B
from combine_router_topk_amd import path as P
from oracle import packed as O

FORMATS = [(c, g, a) for c in (O.INT, O.E2M1) for g in (32, 64, 128) for a in (1, 2)]


def test_a_tile_by_hand():
    """Row 3, column 77 = 32 * 2 + 8 * 1 + 5 lies in lane 16 + 3, its dword 2."""
    assert O.place(3, 77, O.E2M1) == (16 * 19 + 8 + 2, 4)  # nibble 5 of the dword
    assert O.place(3, 77, O.INT) == (16 * 19 + 8 + 1, 4)   # place 5: byte 1, the high half
    q = np.zeros((16, 128), np.uint8)
    q[3, 77] = 11
    b = O.pack(q, np.full((16, 1), 0x3c00, np.uint16), O.E2M1, 128)
    assert b.size == 1056 and b[16 * 19 + 10] == 0xb0 and b[:1024].sum() == 0xb0
    v, mag = O.matrix(b, 16, 128, O.E2M1, 128, 1)
    assert v[3, 77] == -1.5 and np.abs(v).sum() == 1.5 and mag.sum() == 1.5


@pytest.mark.parametrize("codes", [O.INT, O.E2M1])
def test_every_place_is_taken_once(codes):
    seen = {O.place(r, c, codes) for r in range(16) for c in range(128)}
    assert len(seen) == 2048 and {b for b, _ in seen} == set(range(1024)) and {s for _, s in seen} == {0, 4}


@pytest.mark.parametrize("codes,group,act", FORMATS)
@pytest.mark.parametrize("rows,cols", [(1, 8), (16, 128), (40, 200), (33, 264)])
def test_pack_and_back(codes, group, act, rows, cols):
    rng = np.random.default_rng(rows + cols)
    q = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    s = oracle.encode16((rng.random((rows, -(-cols // group))) + 0.5).astype(np.float32), act)
    b = O.pack(q, s, codes, group)
    f = B.make_packed_format(codes, group, act)
    assert b.size == B.moe_packed_weight_bytes(f, 1, rows, cols)
    got, scale = O.unpack(b, rows, cols, codes, group, act)
    assert np.array_equal(got, q)
    assert np.array_equal(scale, np.repeat(oracle.decode16(s, act).astype(np.float64), group, axis=1)[:, :cols])
    v, _ = O.matrix(b, rows, cols, codes, group, act)
    u = P.unpack_weights(torch.from_numpy(b), rows, cols, f)
    assert np.array_equal(u.double().numpy(), v)  # 4 bits by 16 are exact in fp32


@pytest.mark.parametrize("codes,group,act", FORMATS)
def test_packing_takes_the_nearest_code(codes, group, act):
    rng = np.random.default_rng(group)
    w = rng.standard_normal((3, 40, 200)).astype(np.float32)
    w[0, 0, :group] = 0.0
    w[1, 2, 5] = 40.0
    f = B.make_packed_format(codes, group, act)
    b = P.pack_weights(torch.from_numpy(w), f).numpy()
    assert b.shape == (3, B.moe_packed_weight_bytes(f, 1, 40, 200))
    for i in range(3):
        q, s = O.unpack(b[i], 40, 200, codes, group, act)
        v = O.VALUES[codes][q] * s
        grid = np.unique(O.VALUES[codes])
        nearest = np.abs(w[i].astype(np.float64)[..., None] - grid * s[..., None]).min(-1)
        assert (np.abs(v - w[i]) <= nearest + 2e-6 * np.abs(w[i]) + 1e-30).all()
        # the largest of a group takes the largest code, up to the scale's rounding
        top = np.abs(w[i, :, :group]).max(1)
        assert (np.abs(s[:, 0] * (7 if codes == O.INT else 6) - top) <= top * 2.0 ** -8 + 1e-30).all()


def test_packing_refusals():
    f = B.make_packed_format(B.MOE_PACKED_INT, 32, B.MOE_F16)
    with pytest.raises(ValueError, match="not finite"):
        P.pack_weights(torch.full((16, 32), float("nan")), f)
    with pytest.raises(ValueError, match="beyond"):
        P.pack_weights(torch.full((16, 32), 1e6), f)
    with pytest.raises(ValueError, match="rows, cols"):
        P.pack_weights(torch.zeros(16), f)
    assert P.pack_weights(torch.zeros(0, 16, 32), f).shape[0] == 0
