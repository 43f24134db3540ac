"""Weights that are in 4 bits already: their codes and scales come through the layout
unchanged, without a GPU."""
import numpy as np
import pytest
import torch

import oracle
from combine_router_topk_amd import binding as B
from combine_router_topk_amd import path as P
from oracle import packed as O

FORMATS = [(c, g, a) for c in (O.INT, O.E2M1) for g in (32, 64, 128) for a in (B.MOE_F16, B.MOE_BF16)]


def draw(rng, E, rows, cols, codes, group, act):
    """(codes 0 .. 15, what pack_codes takes, scales' bits) as another tool leaves them:
    scales of both signs, some of zero, not tied to the codes' largest."""
    q = rng.integers(0, 16, (E, rows, cols))
    s = rng.standard_normal((E, rows, -(-cols // group))).astype(np.float32)
    s[rng.random(s.shape) < 0.1] = 0
    return q, torch.from_numpy(q - 8 if codes == O.INT else q), oracle.encode16(s, act)


def scales(bits, act):
    return torch.from_numpy(bits.view(np.int16)).view(B._TORCH_ACT[act])


@pytest.mark.parametrize("codes,group,act", FORMATS)
@pytest.mark.parametrize("rows,cols", [(16, 128), (1, 1), (17, 129), (40, 328), (8, 264)])
def test_codes_and_scales_stay_as_they_are(codes, group, act, rows, cols):
    rng = np.random.default_rng(rows + cols)
    q, given, bits = draw(rng, 3, rows, cols, codes, group, act)
    f = B.make_packed_format(codes, group, act)
    got = P.pack_codes(given, scales(bits, act), f)
    assert got.shape == (3, B.moe_packed_weight_bytes(f, 1, rows, cols)) and got.dtype == torch.uint8
    for e in range(3):
        assert np.array_equal(got[e].numpy(), O.pack(q[e], bits[e], codes, group)), e
    want = O.VALUES[codes][q] * np.repeat(oracle.decode16(bits, act), group, 2)[..., :cols]
    assert np.array_equal(P.unpack_weights(got, rows, cols, f).numpy().astype(np.float64), want)


@pytest.mark.parametrize("dtype", [torch.int8, torch.int32, torch.int64])
def test_types_of_codes_and_shapes(dtype):
    f = B.make_packed_format(B.MOE_PACKED_INT, 64, B.MOE_F16)
    c = torch.arange(-8, 8).repeat(2, 3, 16, 5).to(dtype)
    s = torch.rand(2, 3, 16, 2).half()
    got = P.pack_codes(c, s, f)
    assert got.shape == (2, 3, B.moe_packed_weight_bytes(f, 1, 16, 80))
    assert torch.equal(got[1, 2], P.pack_codes(c[1, 2], s[1, 2], f))
    assert torch.equal(P.pack_codes(c.transpose(0, 1), s.transpose(0, 1), f), got.transpose(0, 1))
    few = c.clamp(0, 7)
    assert torch.equal(P.pack_codes(few.to(torch.uint8), s, f), P.pack_codes(few, s, f))
    assert P.pack_codes(c[:0], s[:0], f).shape == (0, 3, got.shape[2])
    e2m1 = B.make_packed_format(B.MOE_PACKED_E2M1, 64, B.MOE_F16)
    assert torch.equal(P.pack_codes((c + 8).to(torch.uint8), s, e2m1), P.pack_codes(c + 8, s, e2m1))


@pytest.mark.parametrize("codes,group,act", FORMATS)
def test_packed_weights_come_back_from_their_own_codes(codes, group, act):
    """What pack_weights made, taken apart and laid out again, is the same bytes."""
    f = B.make_packed_format(codes, group, act)
    w = P.pack_weights(torch.randn(2, 24, 200, generator=torch.Generator().manual_seed(1)), f)
    for m in w:
        q, s = O.unpack(m.numpy(), 24, 200, codes, group, act)
        bits = oracle.encode16(s[:, ::group].astype(np.float32), act)
        assert torch.equal(P.pack_codes(torch.from_numpy(q.astype(np.int64) - (8 if codes == O.INT else 0)), scales(bits, act), f), m)


def test_refusals():
    f = B.make_packed_format(B.MOE_PACKED_INT, 32, B.MOE_F16)
    c, s = torch.zeros(16, 64, dtype=torch.int8), torch.zeros(16, 2, dtype=torch.float16)
    for bad in (c - 9, c + 8, (c + 8).to(torch.uint8), c.long() + (1 << 32)):
        with pytest.raises(ValueError, match="outside -8 .. 7"):
            P.pack_codes(bad, s, f)
    e2m1 = B.make_packed_format(B.MOE_PACKED_E2M1, 32, B.MOE_F16)
    for bad in (c - 1, c + 16):
        with pytest.raises(ValueError, match="outside 0 .. 15"):
            P.pack_codes(bad, s, e2m1)
    with pytest.raises(ValueError, match="whole numbers"):
        P.pack_codes(c.float(), s, f)
    for bad in (s.bfloat16(), s.float(), s[:, :1], s[:8], s[None]):
        with pytest.raises(ValueError, match="scale:"):
            P.pack_codes(c, bad, f)
    for v in (float("nan"), float("inf")):
        with pytest.raises(ValueError, match="not finite"):
            P.pack_codes(c, s + v, f)
    for fmt in (B.make_packed_format(B.MOE_PACKED_INT, 16, B.MOE_F16), B.make_packed_format(5, 32, B.MOE_F16)):
        with pytest.raises(ValueError, match="32, 64 or 128"):
            P.pack_codes(c, s, fmt)
    with pytest.raises(ValueError):
        P.pack_codes(c[0], s[0], f)
    with pytest.raises(ValueError):
        P.pack_codes(c[:, :0], s[:, :0], f)


@pytest.mark.parametrize("codes,group,scale", [(0, 32, B.MOE_F16), (7, 32, B.MOE_F16), (B.MOE_PACKED_INT, 16, B.MOE_F16),
                                               (B.MOE_PACKED_E2M1, 256, B.MOE_F16), (B.MOE_PACKED_INT, 32, B.MOE_F32),
                                               (B.MOE_PACKED_E2M1, 32, 0)])
def test_formats_that_the_calls_refuse_are_not_packed(codes, group, scale):
    """None of them is taken for another one."""
    f = B.make_packed_format(codes, group, scale)
    with pytest.raises(ValueError, match="format"):
        P.pack_weights(torch.ones(16, 128), f)
    with pytest.raises(ValueError, match="format"):
        P.pack_codes(torch.zeros(16, 128, dtype=torch.int8), torch.zeros(16, 4).half(), f)
    with pytest.raises(ValueError, match="format"):
        P.unpack_weights(torch.zeros(1152, dtype=torch.uint8), 16, 128, f)


def test_sizes_are_checked():
    f = B.make_packed_format(B.MOE_PACKED_INT, 32, B.MOE_F16)
    for shape in ((2, 0, 128), (2, 16, 0)):
        with pytest.raises(ValueError, match="rows, cols"):
            P.pack_weights(torch.zeros(shape), f)
    w = P.pack_weights(torch.ones(2, 32, 256), f)
    for rows, cols in ((32, 384), (16, 256), (48, 256), (32, 128), (0, 256)):
        with pytest.raises(ValueError, match="bytes"):
            P.unpack_weights(w, rows, cols, f)
    with pytest.raises(ValueError, match="bytes"):
        P.unpack_weights(w.view(torch.int8), 32, 256, f)
    assert torch.equal(P.unpack_weights(w, 32, 256, f), torch.full((2, 32, 256), 7 * float(np.float16(1 / 7))))
    assert P.unpack_weights(P.pack_weights(torch.zeros(0, 16, 32), f), 16, 32, f).shape == (0, 16, 32)
