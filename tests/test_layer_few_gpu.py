"""The whole layer for a few tokens on the GPU against the oracle, and its
routing against moe_route, bit for bit.

Bounds (u = 2^-24): the gate and up sums are off by at most (H + H / 128 + 8)
2 u of the sum of their terms' magnitudes (a matrix instruction's additions
may truncate); that moves h = round16(v) by a step where v lies that near to
a border, and else not at all. The output's sum adds (I + I / 128 + 24) 2 u a
pair and one rounding."""
import numpy as np
import pytest
import torch

import oracle
from combine_router_topk_amd import binding as B
from layercheck import (ACTS, U, assert_within, bits16, codes8, dev, f64, host, round_bound, scales)
from oracle import layer as L
from pathcheck import say

pytestmark = pytest.mark.gpu


def weights(rng, E, rows, cols, act, kind):
    """(device codes or values, device scales or None, fp64 matrices)"""
    if kind == "e4m3":
        c = codes8(rng, (E, rows, cols))
        s = scales(rng, (E, L.blocks(rows), L.blocks(cols)), 1 / (110 * cols ** 0.5))
        return dev(c), dev(s), np.stack([L.matrix8(c[e], s[e]) for e in range(E)])
    b = bits16(rng, (E, rows, cols), act, cols ** -0.5)
    return dev(b, act), None, oracle.decode16(b, act).astype(np.float64)


def run_layer(p, I, logits, x, wu, su, wd, sd, act):
    out_dt = torch.float32 if p.flags & B.MOE_FLAG_OUT_F32 else dev(x, act).dtype
    idx = torch.full((p.T + 1, p.k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((p.T + 1, p.k), -7.0, device="cuda")
    out = torch.full((p.T + 1, p.H), -7.0, dtype=out_dt, device="cuda")
    ws = torch.full((B.moe_layer_workspace_bytes(p, I),), 255, dtype=torch.uint8, device="cuda")
    B.moe_layer_few_tokens(p, I, dev(logits), dev(x, act), wu, su, wd, sd, idx, w, out, ws)
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


def check_layer(T, E, k, H, I, act, kind, flags=0, logits=None, seed=0):
    say(f"[case] layer T={T} E={E} k={k} H={H} I={I} act={act} {kind} flags={flags}")
    rng = np.random.default_rng(seed + T + E + H)
    p = B.make_problem(T, E, k, H, 1, act, flags)
    if logits is None:
        logits = rng.standard_normal((T, E)).astype(np.float32)
    x = bits16(rng, (T, H), act)
    return check_weights(p, I, logits, x, weights(rng, E, 2 * I, H, act, kind), weights(rng, E, H, I, act, kind), act)


def check_weights(p, I, logits, x, w_up, w_down, act):
    """The layer on these weights, as `weights` gives them, against the oracle."""
    T, k, H, flags = p.T, p.k, p.H, p.flags
    (wu, su, up), (wd, sd, down) = w_up, w_down
    idx, w, out = run_layer(p, I, logits, x, wu, su, wd, sd, act)
    ridx, rw = route(p, logits)
    assert torch.equal(idx, ridx) and torch.equal(w.view(torch.int32), rw.view(torch.int32))
    i, gw = host(idx), host(w).astype(np.float64)
    h, v, want = L.moe_layer(x, i, gw, up, down, act)
    xv = np.abs(oracle.decode16(x, act).astype(np.float64))
    bound = np.zeros_like(want)
    hv = np.abs(oracle.decode16(h, act).astype(np.float64))
    for t in range(T):
        for j in range(k):
            e = i[t, j]
            dz = (H + L.blocks(H) + 8) * 2 * U * (np.abs(up[e]) @ xv[t])
            z = up[e] @ oracle.decode16(x, act)[t].astype(np.float64)
            dv = 1.1 * dz[:I] * np.abs(z[I:]) + np.abs(L.silu(z[:I])) * dz[I:] + 1.1 * dz[:I] * dz[I:] \
                + 8 * U * np.abs(v[t, j])
            lo, hi = (oracle.decode16(oracle.encode16((v[t, j] + d).astype(np.float32), act), act).astype(np.float64)
                      for d in (-dv, dv))
            dh = np.maximum(hi - lo, 0)
            bound[t] += gw[t, j] * (np.abs(down[e]) @ (dh + (I + L.blocks(I) + 24) * 2 * U * (hv[t, j] + dh)))
    got = f64(out)
    if flags & B.MOE_FLAG_OUT_F32:
        assert_within(got, want, bound + 1e-30, "out")
    else:
        assert_within(got, want, bound + round_bound(np.abs(want) + bound, act), "out")
    return out


@pytest.mark.parametrize("kind", ["e4m3", "16 bits"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,E,k,H,I", [(1, 1, 1, 16, 16), (1, 8, 2, 128, 128), (2, 4, 4, 144, 48), (7, 64, 3, 272, 80),
                                       (16, 65, 8, 256, 144), (17, 12, 2, 160, 64), (33, 5, 5, 400, 32),
                                       (64, 7, 3, 96, 112)])
def test_layer(T, E, k, H, I, act, kind):
    check_layer(T, E, k, H, I, act, kind)


@pytest.mark.parametrize("T,E,k,H,I", [(3, 300, 16, 64, 32), (64, 1024, 16, 32, 16), (5, 256, 8, 1040, 528),
                                       (1, 160, 6, 2048, 256)])
def test_layer_many_experts_and_wide_rows(T, E, k, H, I):
    check_layer(T, E, k, H, I, B.MOE_BF16, "e4m3")


class Chosen:
    """The fp64 matrices of some of an operand's experts, made from the GPU's
    codes and scales when they are asked for."""

    def __init__(self, codes, scale):
        self.codes, self.scale, self.shape, self.made = codes, scale, codes.shape, {}

    def __getitem__(self, e):
        if e not in self.made:
            self.made[e] = L.matrix8(self.codes[int(e)].cpu().view(torch.uint8).numpy(), self.scale[int(e)].cpu().numpy())
        return self.made[e]


@pytest.mark.parametrize("T,k,flags", [(33, 2, 0), (64, 4, B.MOE_FLAG_OUT_F32), (7, 10, 0)])
def test_layer_with_a_down_product_in_shares(T, k, flags):
    """More blocks than CUs, unevenly, and weights enough for shares: 257 tiles,
    64 experts of 4112 x 2048; tokens choose among 12 of them."""
    say(f"[case] layer in shares T={T} k={k} flags={flags}")
    E, H, I, act = 64, 4112, 2048, B.MOE_BF16
    rng = np.random.default_rng(T)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T)

    def make(rows, cols):
        c = torch.randint(0, 256, (E, rows, cols), dtype=torch.uint8, device="cuda", generator=gen)
        c &= 0xf7  # no NaN
        s = dev(scales(rng, (E, L.blocks(rows), L.blocks(cols)), 1 / (110 * cols ** 0.5)))
        c = c.view(B.E4M3)
        return c, s, Chosen(c, s)

    logits = rng.standard_normal((T, E)).astype(np.float32)
    logits[:, rng.permutation(E)[:12]] += 20
    p = B.make_problem(T, E, k, H, 1, act, flags)
    assert B.moe_layer_workspace_bytes(p, I) >= 4 * T * H * 4
    check_weights(p, I, logits, bits16(rng, (T, H), act), make(2 * I, H), make(H, I), act)


@pytest.mark.parametrize("kind", ["e4m3", "16 bits"])
@pytest.mark.parametrize("T,E,k,H,I", [(64, 48, 8, 128, 64), (57, 200, 4, 144, 48), (45, 5, 5, 64, 528), (14, 300, 16, 64, 32),
                                       (15, 300, 15, 64, 32)])
def test_layer_around_224_pairs(T, E, k, H, I, kind):
    """From 225 pairs on a block of its own routes, and tiles are taken in turn."""
    check_layer(T, E, k, H, I, B.MOE_F16, kind)


def test_many_pairs_on_two_streams_and_in_a_graph():
    T, E, k, H, I, act = 64, 40, 6, 256, 512, B.MOE_BF16
    rng = np.random.default_rng(12)
    p = B.make_problem(T, E, k, H, 1, act)
    wu, su, _ = weights(rng, E, 2 * I, H, act, "e4m3")
    wd, sd, _ = weights(rng, E, H, I, act, "e4m3")
    logits = [rng.standard_normal((T, E)).astype(np.float32) for _ in range(2)]
    x = [bits16(rng, (T, H), act) for _ in range(2)]
    want = [run_layer(p, I, lg, xx, wu, su, wd, sd, act) for lg, xx in zip(logits, x)]
    ins = [(dev(lg), dev(xx, act)) for lg, xx in zip(logits, x)]
    outs = [(torch.empty_like(want[0][0]), torch.empty_like(want[0][1]), torch.empty_like(want[0][2]),
             torch.full((B.moe_layer_workspace_bytes(p, I),), 255, dtype=torch.uint8, device="cuda")) for _ in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]

    def call(i, stream=None):
        B.moe_layer_few_tokens(p, I, *ins[i], wu, su, wd, sd, *outs[i], stream)

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
    for turn in range(4):
        for t in outs[0][:3]:
            t.zero_()
        call(1)
        graph.replay()
        torch.cuda.synchronize()
        check(0), check(1)


@pytest.mark.parametrize("kind", ["e4m3", "16 bits"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,E,k,H,I", [(2, 16, 3, 4096, 48), (20, 6, 2, 4112, 32), (40, 4, 2, 4240, 16)])
def test_layer_rows_of_256_blocks_and_more(T, E, k, H, I, act, kind):
    """The down product's blocks take 8 waves from 256 on, 16 below."""
    check_layer(T, E, k, H, I, act, kind)


def test_layer_fp32_output():
    check_layer(9, 8, 2, 144, 80, B.MOE_F16, "e4m3", B.MOE_FLAG_OUT_F32)
    check_layer(40, 8, 2, 144, 80, B.MOE_BF16, "16 bits", B.MOE_FLAG_OUT_F32)


@pytest.mark.parametrize("act", ACTS)
def test_swiglu_over_all_gates(act):
    """Gates that are exact beside an up value of 2^60 (fp16: 1) that shows
    silu where exp(-gate) is no fp32 number any more; the down product picks
    one inner value. The bound is the inner value's rounding, 8 u of silu and
    half of fp32's last step."""
    say(f"[case] SwiGLU over all gates act={act}")
    I, H, E, T = 32, 32, 1, 64
    up = 1.0 if act == B.MOE_F16 else 2.0 ** 60
    gates = np.concatenate([np.linspace(-120, -60, 61), [0.0, 90.0, 448.0]])
    x = np.zeros((T, H), np.float32)
    x[:, 0], x[:, 1] = gates, 1.0
    wu, wd = np.zeros((E, 2 * I, H), np.float32), np.zeros((E, H, I), np.float32)
    wu[0, :I, 0], wu[0, I:, 1] = 1.0, up
    wd[0, :, 3] = 1.0
    bits = lambda a: dev(oracle.encode16(a, act), act)  # noqa: E731
    p = B.make_problem(T, E, 1, H, 1, act, B.MOE_FLAG_OUT_F32)
    _, w, out = run_layer(p, I, np.zeros((T, E), np.float32), oracle.encode16(x, act), bits(wu), None, bits(wd), None,
                          act)
    g = oracle.decode16(oracle.encode16(x, act), act)[:, 0].astype(np.float64)
    v = np.repeat((L.silu(g) * up)[:, None], H, axis=1)
    assert (w == 1.0).all()
    near = 8 * U * np.abs(v) + 2.0 ** -150 * up
    assert_within(f64(out), v, near + round_bound(np.abs(v) + near, act), "out")


@pytest.mark.parametrize("act", ACTS)
def test_swiglu_at_gates_to_the_end_of_fp32(act):
    """Gates down to nearly -FLT_MAX, where -gate log2(e) is no fp32 number any
    more: silu is -0 and the output 0, exactly."""
    say(f"[case] SwiGLU at gates to the end of fp32 act={act}")
    I, H, E = 128, 16, 1
    gates = np.array([-2.0 ** -14, -0.5, -1.0, -1.25, -1.375, -1.390625, -1.5, -1.75, -1.9921875], np.float32)
    T = len(gates)
    x = np.zeros((T, H), np.float32)
    x[:, 0], x[:, 1] = gates, 1.0
    wu, wd = np.zeros((E, 2 * I, H), np.uint8), np.zeros((E, H, I), np.uint8)
    wu[0, :I, 0], wu[0, I:, 1], wd[0, :, 3] = 0x38, 0x38, 0x38
    su = np.array([2.0 ** 127, 1.0], np.float32).reshape(E, 2, 1)
    p = B.make_problem(T, E, 1, H, 1, act, B.MOE_FLAG_OUT_F32)
    _, _, out = run_layer(p, I, np.zeros((T, E), np.float32), oracle.encode16(x, act), dev(wu), dev(su), dev(wd),
                          dev(np.ones((E, 1, 1), np.float32)), act)
    assert (out == 0).all(), out[:, 0]


def test_every_token_on_one_expert():
    T, E = 64, 9
    logits = np.zeros((T, E), np.float32)
    logits[:, 5] = 3.0
    check_layer(T, E, 1, 128, 64, B.MOE_BF16, "e4m3", logits=logits)


def test_ties_nan_and_infinite_logits_route_as_the_router_does():
    rng = np.random.default_rng(3)
    for E, k in ((16, 5), (100, 7), (256, 8), (1000, 16)):
        T = 24
        logits = rng.integers(-2, 3, (T, E)).astype(np.float32)
        logits[1], logits[2] = 0.0, np.nan
        logits[3, ::2], logits[4, 3], logits[5, 1] = np.nan, np.inf, -np.inf
        logits[6] = -0.0
        logits[7] = -np.inf
        H, I, act = 32, 16, B.MOE_F16
        p = B.make_problem(T, E, k, H, 1, act)
        x = bits16(rng, (T, H), act)
        wu, su, _ = weights(rng, E, 2 * I, H, act, "e4m3")
        wd, sd, _ = weights(rng, E, H, I, act, "e4m3")
        idx, w, out = run_layer(p, I, logits, x, wu, su, wd, sd, act)
        ridx, rw = route(p, logits)
        assert torch.equal(idx, ridx), (E, k)
        assert torch.equal(w.view(torch.int32), rw.view(torch.int32)), (E, k)
        # a token whose weights are NaN has a NaN output, the others have not
        nan = torch.isnan(w).any(dim=1)
        assert torch.isnan(out[nan]).all() and not torch.isnan(out[~nan]).any(), (E, k)


def test_non_finite_tokens_stay_their_own():
    T, E, k, H, I, act = 20, 6, 2, 160, 48, B.MOE_BF16
    rng = np.random.default_rng(4)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    x = bits16(rng, (T, H), act)
    wu, su, _ = weights(rng, E, 2 * I, H, act, "e4m3")
    wd, sd, _ = weights(rng, E, H, I, act, "e4m3")
    p = B.make_problem(T, E, k, H, 1, act)
    _, _, want = run_layer(p, I, logits, x, wu, su, wd, sd, act)
    x2 = x.copy()
    x2[3, H - 1], x2[17, 0] = 0x7fc0, 0x7f80  # a NaN, an infinity
    _, _, got = run_layer(p, I, logits, x2, wu, su, wd, sd, act)
    rest = [t for t in range(T) if t not in (3, 17)]
    assert torch.equal(got[rest], want[rest]) and torch.isnan(got[3]).all() and not torch.isfinite(got[17]).all()


def test_layer_repeats_bit_for_bit_and_takes_a_stream():
    T, E, k, H, I, act = 40, 32, 4, 512, 256, B.MOE_BF16
    rng = np.random.default_rng(6)
    logits, x = rng.standard_normal((T, E)).astype(np.float32), bits16(rng, (T, H), act)
    wu, su, _ = weights(rng, E, 2 * I, H, act, "e4m3")
    wd, sd, _ = weights(rng, E, H, I, act, "e4m3")
    p = B.make_problem(T, E, k, H, 1, act)
    first = run_layer(p, I, logits, x, wu, su, wd, sd, act)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = run_layer(p, I, logits, x, wu, su, wd, sd, act)
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_no_tokens():
    p = B.make_problem(0, 8, 2, 64, 1, B.MOE_BF16)
    B.moe_layer_few_tokens(p, 64, *(None,) * 10)
