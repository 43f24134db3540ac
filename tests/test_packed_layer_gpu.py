"""The whole layer for a few tokens with 4-bit weights on the GPU against the
oracle, and its routing against moe_route, bit for bit.

Bounds (u = 2^-24): a sum of n terms is off by at most (n + n / 32 + 8) 2 u of
the magnitudes of what is summed (products, with integer codes those of 0 .. 15
and of 8; a matrix instruction's additions may truncate; a scaling each 32 columns
or more). That moves h = round16(v) by a step where v lies that near to a border,
and else not at all. The output's sum adds (I + I / 32 + 24) 2 u a pair and one
rounding."""
import numpy as np
import pytest
import torch

import oracle
from combine_router_topk_amd import binding as B
from combine_router_topk_amd import path as P
from layercheck import ACTS, U, assert_within, bits16, dev, f64, host, round_bound
from oracle import layer as L
from oracle import packed as O
from packedcheck import FORMATS, Weights
from pathcheck import say

pytestmark = pytest.mark.gpu


def run_layer(p, logits, x, wu, wd, act):
    out_dt = torch.float32 if p.flags & B.MOE_FLAG_OUT_F32 else dev(x, act).dtype
    I = wd.cols
    idx = torch.full((p.T + 1, p.k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((p.T + 1, p.k), -7.0, device="cuda")
    out = torch.full((p.T + 1, p.H), -7.0, dtype=out_dt, device="cuda")
    ws = torch.full((B.moe_layer_packed_workspace_bytes(p, I),), 255, dtype=torch.uint8, device="cuda")
    B.moe_layer_few_tokens_packed(p, wu.format, I, dev(logits), dev(x, act), wu.dev, wd.dev, idx, w, out, ws)
    torch.cuda.synchronize()
    assert (idx[p.T] == -7).all() and (w[p.T] == -7).all() and (out[p.T] == -7).all()
    return idx[:p.T], w[:p.T], out[:p.T]


def route(p, logits):
    idx = torch.empty(p.T, p.k, dtype=torch.int32, device="cuda")
    w = torch.empty(p.T, p.k, device="cuda")
    counts = torch.empty(p.E, dtype=torch.int32, device="cuda")
    ws = torch.empty(B.moe_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    B.moe_route(p, dev(logits), idx, w, counts, ws)
    return idx, w


def inner_bounds(z, dz, I):
    """How far silu(gate) up may be off where the sums z are off by dz."""
    g, u, dg, du = z[..., :I], z[..., I:], dz[..., :I], dz[..., I:]
    v = L.silu(g) * u
    return v, 1.1 * dg * np.abs(u) + np.abs(L.silu(g)) * du + 1.1 * dg * du + 8 * U * np.abs(v)


def check_layer(T, E, k, H, I, act, codes, group, flags=0, logits=None, scale_act=None, seed=0):
    say(f"[case] packed layer T={T} E={E} k={k} H={H} I={I} act={act} codes={codes} group={group} flags={flags}")
    rng = np.random.default_rng(seed + T + E + H)
    p = B.make_problem(T, E, k, H, 1, act, flags)
    if logits is None:
        logits = rng.standard_normal((T, E)).astype(np.float32)
    x = bits16(rng, (T, H), act)
    wu = Weights(rng, E, 2 * I, H, codes, group, scale_act or act)
    wd = Weights(rng, E, H, I, codes, group, scale_act or act)
    idx, w, out = run_layer(p, logits, x, wu, wd, act)
    ridx, rw = route(p, logits)
    assert torch.equal(idx, ridx) and torch.equal(w.view(torch.int32), rw.view(torch.int32))
    i, gw = host(idx), host(w).astype(np.float64)
    xv = oracle.decode16(x, act).astype(np.float64)
    to16 = lambda a: oracle.decode16(oracle.encode16(a.astype(np.float32), act), act).astype(np.float64)  # noqa: E731
    want, bound = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            up, mag = wu.both(i[t, j])
            v, dv = inner_bounds(up @ xv[t], (H + H / 32 + 8) * 2 * U * (mag @ np.abs(xv[t])), I)
            h = to16(v)
            dh = np.maximum(to16(v + dv) - to16(v - dv), 0)
            down, mag = wd.both(i[t, j])
            want[t] += gw[t, j] * (down @ h)
            bound[t] += gw[t, j] * (np.abs(down) @ dh + (I + I / 32 + 24) * 2 * U * (mag @ (np.abs(h) + dh)))
    if flags & B.MOE_FLAG_OUT_F32:
        assert_within(f64(out), want, bound + 1e-30, "out")
    else:
        assert_within(f64(out), want, bound + round_bound(np.abs(want) + bound, act), "out")
    return out


@pytest.mark.parametrize("codes,group", FORMATS)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,E,k,H,I", [(1, 1, 1, 16, 16), (1, 8, 2, 128, 128), (2, 4, 4, 144, 48), (7, 64, 3, 272, 80),
                                       (16, 65, 8, 256, 144), (17, 12, 2, 160, 64), (33, 5, 5, 400, 32),
                                       (64, 7, 3, 96, 112)])
def test_layer(T, E, k, H, I, act, codes, group):
    check_layer(T, E, k, H, I, act, codes, group)


@pytest.mark.parametrize("T,E,k,H,I", [(3, 300, 16, 64, 32), (64, 1024, 16, 32, 16), (5, 256, 8, 1040, 528),
                                       (1, 160, 6, 2048, 256), (64, 48, 8, 128, 64), (57, 200, 4, 144, 48),
                                       (14, 300, 16, 64, 32), (15, 300, 15, 64, 32), (2, 16, 3, 4096, 48), (20, 6, 2, 4112, 32)])
def test_layer_many_experts_wide_rows_and_around_224_pairs(T, E, k, H, I):
    check_layer(T, E, k, H, I, B.MOE_BF16, O.INT, 128)
    check_layer(T, E, k, H, I, B.MOE_F16, O.E2M1, 32)


@pytest.mark.parametrize("T,E,k,H,I", [(64, 128, 8, 144, 176), (28, 256, 8, 144, 400)])
def test_layer_of_many_tiles(T, E, k, H, I):
    """Blocks of two pairs of tiles, the last one of an expert without its second."""
    check_layer(T, E, k, H, I, B.MOE_BF16, O.INT, 128)
    check_layer(T, E, k, H, I, B.MOE_F16, O.E2M1, 32)


@pytest.mark.parametrize("codes,group", FORMATS)
def test_layer_fp32_output_and_scales_of_the_other_format(codes, group):
    check_layer(9, 8, 2, 144, 80, B.MOE_F16, codes, group, B.MOE_FLAG_OUT_F32, scale_act=B.MOE_BF16)
    check_layer(40, 8, 2, 144, 80, B.MOE_BF16, codes, group, B.MOE_FLAG_OUT_F32, scale_act=B.MOE_F16)


def test_every_token_on_one_expert():
    logits = np.zeros((64, 9), np.float32)
    logits[:, 5] = 3.0
    check_layer(64, 9, 1, 128, 64, B.MOE_BF16, O.INT, 64, logits=logits)


@pytest.mark.parametrize("T,k,flags", [(33, 2, 0), (64, 4, B.MOE_FLAG_OUT_F32), (7, 10, 0)])
def test_layer_with_a_down_product_in_shares(T, k, flags):
    """More blocks than CUs, unevenly, and weights enough for shares: 257 tiles, 128
    experts of 4112 x 2048; tokens choose among 12 of them."""
    rng = np.random.default_rng(T)
    E = 128
    logits = rng.standard_normal((T, E)).astype(np.float32)
    logits[:, rng.permutation(E)[:12]] += 20
    check_layer(T, E, k, 4112, 2048, B.MOE_BF16, O.E2M1, 64, flags, logits)


@pytest.mark.parametrize("T,k,H,I,flags", [(64, 1, 2064, 1024, 0), (11, 6, 2064, 1040, B.MOE_FLAG_OUT_F32),
                                           (9, 8, 16, 131072, 0)])
def test_layer_in_shares_of_few_tiles(T, k, H, I, flags):
    """An odd number of tiles, fewer than CUs, one with the inner rows alone."""
    rng = np.random.default_rng(T)
    E = 65
    logits = rng.standard_normal((T, E)).astype(np.float32)
    logits[:, rng.permutation(E)[:9]] += 20
    check_layer(T, E, k, H, I, B.MOE_F16, O.INT, 32, flags, logits)


def test_ties_nan_and_infinite_logits_route_as_the_router_does():
    rng = np.random.default_rng(3)
    for E, k in ((16, 5), (100, 7), (256, 8), (1000, 16)):
        T = 24
        logits = rng.integers(-2, 3, (T, E)).astype(np.float32)
        logits[1], logits[2] = 0.0, np.nan
        logits[3, ::2], logits[4, 3], logits[5, 1] = np.nan, np.inf, -np.inf
        logits[6], logits[7] = -0.0, -np.inf
        H, I, act = 32, 16, B.MOE_F16
        p = B.make_problem(T, E, k, H, 1, act)
        x = bits16(rng, (T, H), act)
        wu, wd = Weights(rng, E, 2 * I, H, O.INT, 32, act), Weights(rng, E, H, I, O.INT, 32, act)
        idx, w, out = run_layer(p, logits, x, wu, wd, act)
        ridx, rw = route(p, logits)
        assert torch.equal(idx, ridx) and torch.equal(w.view(torch.int32), rw.view(torch.int32)), (E, k)
        nan = torch.isnan(w).any(dim=1)
        assert torch.isnan(out[nan]).all() and not torch.isnan(out[~nan]).any(), (E, k)


@pytest.mark.parametrize("codes", [O.INT, O.E2M1])
def test_non_finite_tokens_stay_their_own(codes):
    T, E, k, H, I, act = 20, 6, 2, 160, 48, B.MOE_BF16
    rng = np.random.default_rng(4)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    x = bits16(rng, (T, H), act)
    wu, wd = Weights(rng, E, 2 * I, H, codes, 64, act), Weights(rng, E, H, I, codes, 64, act)
    p = B.make_problem(T, E, k, H, 1, act)
    _, _, want = run_layer(p, logits, x, wu, wd, act)
    x2 = x.copy()
    x2[3, H - 1], x2[17, 0] = 0x7fc0, 0x7f80  # a NaN, an infinity
    _, _, got = run_layer(p, logits, x2, wu, wd, act)
    rest = [t for t in range(T) if t not in (3, 17)]
    assert torch.equal(got[rest], want[rest]) and torch.isnan(got[3]).all() and not torch.isfinite(got[17]).all()


def test_two_streams_and_a_graph():
    T, E, k, H, I, act = 64, 40, 6, 256, 512, B.MOE_BF16
    rng = np.random.default_rng(12)
    p = B.make_problem(T, E, k, H, 1, act)
    wu, wd = Weights(rng, E, 2 * I, H, O.INT, 128, act), Weights(rng, E, H, I, O.INT, 128, act)
    logits = [rng.standard_normal((T, E)).astype(np.float32) for _ in range(2)]
    x = [bits16(rng, (T, H), act) for _ in range(2)]
    want = [run_layer(p, lg, xx, wu, wd, act) for lg, xx in zip(logits, x)]
    ins = [(dev(lg), dev(xx, act)) for lg, xx in zip(logits, x)]
    outs = [(*(torch.empty_like(t) for t in want[0]),
             torch.full((B.moe_layer_packed_workspace_bytes(p, I),), 255, dtype=torch.uint8, device="cuda"))
            for _ in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]

    def call(i, stream=None):
        B.moe_layer_few_tokens_packed(p, wu.format, I, *ins[i], wu.dev, wd.dev, *outs[i], stream)

    def check(i):
        for a, b in zip(outs[i], want[i]):
            assert torch.equal(a, b), i

    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            call(i, streams[i])
    torch.cuda.synchronize()
    check(0), check(1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0)
    for _ in range(4):
        for t in outs[0][:3]:
            t.zero_()
        call(1)
        graph.replay()
        torch.cuda.synchronize()
        check(0), check(1)


def test_path_packs_and_runs():
    """Packing, the layer for a few tokens and the layer through the products agree
    with each other to the bounds' size."""
    T, E, k, H, I, act = 32, 16, 4, 256, 128, B.MOE_F16
    torch.manual_seed(0)
    f = B.make_packed_format(B.MOE_PACKED_INT, 64, act)
    w = P.pack_experts(torch.randn(E, 2 * I, H, device="cuda") / H ** 0.5, torch.randn(E, H, I, device="cuda") / I ** 0.5, f)
    p = B.make_problem(T, E, k, H, 1, act)
    b = P.allocate(p, torch.randn(T, E), torch.randn(T, H).half())
    P.layer_few_tokens_packed(b, w, P.layer_packed_workspace(b, I))
    few = b.out.float().clone()
    P.run_layer_packed(b, w, torch.empty(T * k, I, dtype=torch.float16, device="cuda"))
    torch.cuda.synchronize()
    up, down = P.unpack_weights(w.w_up, 2 * I, H, f), P.unpack_weights(w.w_down, H, I, f)
    for t in (0, 13):
        z = torch.stack([up[e] @ b.x[t].float() for e in b.idx.view(T, k)[t].tolist()])
        h = torch.nn.functional.silu(z[:, :I]) * z[:, I:]
        y = torch.stack([down[e] @ hh for e, hh in zip(b.idx.view(T, k)[t].tolist(), h)])
        want = (b.w.view(T, k)[t][:, None] * y).sum(0)
        # h, y and out are rounded to fp16; fp32 sums of up to 272 terms on both sides
        gate = b.w.view(T, k)[t][:, None]
        size = torch.stack([down[e].abs() @ hh.abs() for e, hh in zip(b.idx.view(T, k)[t].tolist(), h)])
        tol = 2.0 ** -11 * ((gate * size).sum(0) + (gate * y.abs()).sum(0) + want.abs()) * 1.01 \
            + 2 * 300 * 2 * U * (gate * size).sum(0) * 4 + 2.0 ** -20
        assert ((few[t] - want).abs() <= tol).all() and ((b.out[t].float() - want).abs() <= tol).all()


def test_no_tokens():
    p = B.make_problem(0, 8, 2, 64, 1, B.MOE_BF16)
    B.moe_layer_few_tokens_packed(p, B.make_packed_format(1, 32, 1), 64, *(None,) * 8)
