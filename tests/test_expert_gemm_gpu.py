"""The experts' products in 8 bits on the GPU against the oracle.

Bounds (u = 2^-24). 8-bit matrix instructions, which bf16 outputs come from,
sum groups of eight products cut off at 2^-13 of a power of two that the
largest of them reaches: at most 8 2^-13 of the group's largest product is
lost, with rounded fp32 sums of the groups and blocks after that. fp16 and fp32
outputs, bf16 ones with exact sums and the SwiGLU's come from products in fp16,
exact, summed in fp32 with at most K + K / 128 + 2 truncations.
"""
import numpy as np
import pytest
import torch

from combine_router_topk_amd import binding as B
from layercheck import (ACTS, HALF, U, assert_within, check_rows8, codes8, codes_of, dev, f64, round_bound, scales)
from oracle import layer as L
from pathcheck import say

pytestmark = pytest.mark.gpu


def routed(rng, T, E, k, shape="even"):
    """src, counts, offsets of a batch whose experts are in a shuffled order
    of ranks, as a layout over several ranks gives them."""
    p = np.ones(E)
    if shape == "skewed":
        p = 1.0 / np.arange(1, E + 1) ** 2
    if shape == "few":
        p[: E - max(k, 1)] = 1e-12
    keys = np.log(p) + rng.gumbel(size=(T, E))
    idx = np.argsort(-keys, axis=1)[:, :k]
    order = rng.permutation(E)
    place = np.empty(E, np.int64)
    place[order] = np.arange(E)
    src = np.argsort(place[idx.ravel()], kind="stable").astype(np.int32)
    counts = np.bincount(idx.ravel(), minlength=E)
    offsets = np.zeros(E, np.int64)
    offsets[order] = np.cumsum(counts[order]) - counts[order]
    return src, counts.astype(np.int32), offsets.astype(np.int32)


def inputs(rng, T, E, k, K, N, gather, shape="even"):
    src, counts, offsets = routed(rng, T, E, k, shape)
    rows = T if gather else T * k
    a, w = codes8(rng, (rows, K)), codes8(rng, (E, N, K))
    sa = scales(rng, (rows, L.blocks(K)), 1 / 110)
    sw = scales(rng, (E, L.blocks(N), L.blocks(K)), 1 / (110 * K ** 0.5))
    return a, sa, src if gather else None, w, sw, counts, offsets


def run_gemm(T, E, k, K, N, inp, act, flags=0, rows_after=2):
    p = B.make_problem(T, E, k, 8, 1, act, flags)
    dt = torch.float32 if flags else dev(np.zeros(1, np.uint16), act).dtype
    y = torch.full((T * k + rows_after, N), 7.0, dtype=dt, device="cuda")
    B.moe_expert_gemm(p, K, N, *(dev(i) for i in inp), y)
    torch.cuda.synchronize()
    assert (y[T * k:] == 7.0).all()
    return y[:T * k]


def lost_in_groups(inp, k, rows, N):
    """8 2^-13 of the largest product of every group of eight, summed."""
    a, sa, src, w, sw, counts, offsets = inp
    K = a.shape[1]
    out = np.zeros((rows, N))
    for e, r in L.segments(counts, offsets, rows):
        rr = r if src is None else src[r] // k
        av, wv = np.abs(L.values8(a[rr], sa[rr])), np.abs(L.matrix8(w[e], sw[e]))
        for lo in range(0, K, 8):
            m = np.zeros((len(r), N))
            for c in range(lo, min(K, lo + 8)):
                np.maximum(m, np.outer(av[:, c], wv[:, c]), out=m)
            out[r] += 2.0 ** -10 * m
    return out


SHAPES = [  # T, E, k, K, N
    (1, 1, 1, 16, 8), (1, 4, 2, 128, 264), (3, 4, 2, 144, 136), (70, 5, 2, 272, 520), (130, 3, 1, 512, 256),
    (257, 2, 1, 640, 40), (90, 8, 4, 400, 24), (40, 300, 3, 128, 16), (33, 1024, 16, 48, 8)]


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("T,E,k,K,N", SHAPES)
def test_product(T, E, k, K, N, gather):
    rng = np.random.default_rng(T + K)
    inp = inputs(rng, T, E, k, K, N, gather)
    y, mag = L.expert_gemm(*inp[:3], k, *inp[3:], T * k)
    for act in ACTS:
        say(f"[case] product T={T} E={E} k={k} K={K} N={N} gather={gather} act={act}")
        got = run_gemm(T, E, k, K, N, inp, act)
        bound = lost_in_groups(inp, k, T * k, N) + (K // 8 + 2 * L.blocks(K) + 2) * 2 * U * mag
        assert_within(f64(got), y, bound + round_bound(np.abs(y) + bound, act), "y")
    got = run_gemm(T, E, k, K, N, inp, B.MOE_BF16, B.MOE_FLAG_OUT_F32)
    assert_within(f64(got), y, (K + L.blocks(K) + 4) * 2 * U * mag, "y in fp32")


@pytest.mark.parametrize("shape", ["skewed", "few"])
@pytest.mark.parametrize("T,E,k,K,N", [(700, 6, 2, 256, 136), (1100, 3, 1, 144, 72), (520, 40, 4, 128, 264)])
def test_product_uneven_segments(T, E, k, K, N, shape):
    say(f"[case] product {shape} T={T} E={E} k={k} K={K} N={N}")
    rng = np.random.default_rng(T)
    for gather in (True, False):
        inp = inputs(rng, T, E, k, K, N, gather, shape)
        y, mag = L.expert_gemm(*inp[:3], k, *inp[3:], T * k)
        got = run_gemm(T, E, k, K, N, inp, B.MOE_BF16, B.MOE_FLAG_OUT_F32)
        assert_within(f64(got), y, (K + L.blocks(K) + 4) * 2 * U * mag, "y in fp32")
        got = run_gemm(T, E, k, K, N, inp, B.MOE_BF16)
        bound = lost_in_groups(inp, k, T * k, N) + (K // 8 + 2 * L.blocks(K) + 2) * 2 * U * mag
        assert_within(f64(got), y, bound + round_bound(np.abs(y) + bound, B.MOE_BF16), "y")


def swiglu_bounds(inp, T, k, K, I):
    """v and how far fp32 sums may be off: |silu'| is at most 1.1, and exp,
    the division and two products add under 8 u."""
    z, mag = L.expert_gemm(*inp[:3], k, *inp[3:], T * k)
    dz = (K + L.blocks(K) + 4) * 2 * U * mag
    g, u = z[:, :I], z[:, I:]
    v = L.silu(g) * u
    dg, du = dz[:, :I], dz[:, I:]
    dv = 1.1 * dg * np.abs(u) + np.abs(L.silu(g)) * du + 1.1 * dg * du + 8 * U * np.abs(v)
    return v, dv


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("T,E,k,K,I", [(1, 1, 1, 16, 16), (1, 4, 2, 128, 128), (3, 4, 2, 144, 144), (70, 5, 2, 272, 80),
                                       (130, 3, 1, 512, 256), (257, 2, 1, 640, 32), (700, 6, 2, 256, 208)])
def test_swiglu(T, E, k, K, I, gather):
    say(f"[case] SwiGLU T={T} E={E} k={k} K={K} I={I} gather={gather}")
    rng = np.random.default_rng(T + I)
    inp = inputs(rng, T, E, k, K, 2 * I, gather, "skewed" if T > 500 else "even")
    n, nb = T * k, L.blocks(I)
    q = torch.full((n + 2, I), 7.0, device="cuda").to(B.E4M3)
    s = torch.full((n + 2, nb), 7.0, device="cuda")
    B.moe_expert_gemm_swiglu(B.make_problem(T, E, k, 8, 1, B.MOE_BF16), K, I, *(dev(i) for i in inp), q, s)
    torch.cuda.synchronize()
    v, dv = swiglu_bounds(inp, T, k, K, I)
    check_rows8(codes_of(q[:n]), f64(s[:n]), v, dv, "q")
    assert (q[n:].float() == 7.0).all() and (s[n:] == 7.0).all()


def test_swiglu_over_all_gates():
    """Gates that are exact (one code times powers of two, and 1.5) and beside
    an up value of 2^60 that shows silu where exp(-gate) is no fp32 number any
    more: 8 u of its value, and half of fp32's last step of 2^-149."""
    say("[case] SwiGLU over all gates")
    E, K, I, up = 128, 16, 128, 2.0 ** 60
    gate_codes = np.arange(256, dtype=np.uint8)[[c for c in range(256) if c & 127 != 127]]
    sa = np.array([1.0, 1.5, 0.25, 2.0 ** -20, 2.0 ** -60], np.float32)
    for part in (gate_codes[:127], gate_codes[127:]):
        E, T = len(part), len(part) * len(sa)
        a, w = np.zeros((T, K), np.uint8), np.zeros((E, 2 * I, K), np.uint8)
        a[:, 0], w[:, :I, 0], w[:, I:, 0] = 0x38, part[:, None], 0x38
        sw = np.broadcast_to(np.array([1.0, up], np.float32)[:, None], (E, 2, 1)).copy()
        counts, offsets = np.full(E, len(sa), np.int32), np.arange(E, dtype=np.int32) * len(sa)
        rows = np.tile(sa, E)
        q, s = torch.empty(T, I, device="cuda").to(B.E4M3), torch.empty(T, 1, device="cuda")
        B.moe_expert_gemm_swiglu(B.make_problem(T, E, 1, 8, 1, B.MOE_BF16), K, I,
                                 *(dev(i) for i in (a, rows[:, None].copy(), None, w, sw, counts, offsets)), q, s)
        torch.cuda.synchronize()
        z = np.repeat(L.decode8(part), len(sa)) * rows
        v = np.repeat((L.silu(z) * up * rows)[:, None], I, axis=1)
        check_rows8(codes_of(q), f64(s), v, 8 * U * np.abs(v) + 2.0 ** -150 * up * rows[:, None], "q")


def test_swiglu_at_gates_to_the_end_of_fp32():
    """Gates that are exact, down to -FLT_MAX, where -gate log2(e) is no fp32
    number any more and silu is -0. They spoil nothing of their block, whose
    other gates are positive (2^-9 of the magnitude: silu is the gate), beside
    up values of 2^-120 of it."""
    say("[case] SwiGLU at gates to the end of fp32")
    far = np.array([1e5, 1e20, 1e30, 2.3e38, 2.36e38, 2.4e38, 3e38, np.finfo(np.float32).max], np.float32)
    T, K, I, up = len(far), 16, 128, 2.0 ** -120
    a, w = np.zeros((T, K), np.uint8), np.zeros((1, 2 * I, K), np.uint8)
    a[:, 0], w[0, :I, 0], w[0, I:, 0] = 0x38, 0x01, 0x38  # 1, 2^-9, 1
    w[0, [0, 77], 0] = 0xb8                               # -1
    sw = np.array([1.0, up], np.float32).reshape(1, 2, 1)
    inp = (a, far[:, None].copy(), None, w, sw, np.array([T], np.int32), np.zeros(1, np.int32))
    q, s = torch.empty(T, I, device="cuda").to(B.E4M3), torch.empty(T, 1, device="cuda")
    B.moe_expert_gemm_swiglu(B.make_problem(T, 1, 1, 8, 1, B.MOE_BF16), K, I, *(dev(i) for i in inp), q, s)
    torch.cuda.synchronize()
    z = L.decode8(w[0, :, 0])[None] * far[:, None].astype(np.float64)
    v = L.silu(z[:, :I]) * z[:, I:] * up
    assert torch.isfinite(s).all(), s
    check_rows8(codes_of(q), f64(s), v, 8 * U * np.abs(v), "q")


def test_neighbours_do_not_leak():
    """NaN in the rows, the columns and the experts beside those a result is
    made of, where loads past the end of K, of N or of a segment would meet
    it."""
    say("[case] NaN beside every segment")
    T, E, k, K, N = 70, 3, 1, 144, 136
    rng = np.random.default_rng(11)
    a, sa, _, w, sw, counts, offsets = inputs(rng, T, E, k, K, N, False)
    e = int(np.argmax(counts))
    nan_e = [i for i in range(E) if i != e]
    a2, w2, sa2, sw2 = a.copy(), w.copy(), sa.copy(), sw.copy()
    mine = np.arange(offsets[e], offsets[e] + counts[e])
    others = np.setdiff1d(np.arange(T), mine)
    a2[others], sa2[others], w2[nan_e], sw2[nan_e] = 0x7f, np.nan, 0x7f, np.nan
    for flags in (0, B.MOE_FLAG_OUT_F32):
        want = run_gemm(T, E, k, K, N, (a, sa, None, w, sw, counts, offsets), B.MOE_BF16, flags)
        got = run_gemm(T, E, k, K, N, (a2, sa2, None, w2, sw2, counts, offsets), B.MOE_BF16, flags)
        assert torch.equal(got[mine], want[mine]) and torch.isnan(got[others]).all()
        # one NaN code in a row, in its last columns
        a3 = a.copy()
        a3[mine[0], K - 1] = 0xff
        got = run_gemm(T, E, k, K, N, (a3, sa, None, w, sw, counts, offsets), B.MOE_BF16, flags)
        assert torch.isnan(got[mine[0]]).all() and torch.equal(got[mine[1:]], want[mine[1:]])
        # one NaN code in a weight row: its column of its expert
        w3 = w.copy()
        w3[e, N - 1, K - 16] = 0x7f
        got = run_gemm(T, E, k, K, N, (a, sa, None, w3, sw, counts, offsets), B.MOE_BF16, flags)
        assert torch.isnan(got[mine, N - 1]).all() and torch.equal(got[:, :N - 1], want[:, :N - 1])
        assert torch.equal(got[others], want[others])


def test_swiglu_non_finite():
    say("[case] SwiGLU with a NaN row and an infinite scale")
    T, E, k, K, I = 20, 2, 1, 144, 144
    rng = np.random.default_rng(12)
    a, sa, _, w, sw, counts, offsets = inputs(rng, T, E, k, K, 2 * I, False)
    sa[3, 0], sa[5, 1] = np.nan, np.inf
    q, s = torch.empty(T, I, device="cuda").to(B.E4M3), torch.empty(T, 2, device="cuda")
    B.moe_expert_gemm_swiglu(B.make_problem(T, E, k, 8, 1, B.MOE_BF16), K, I,
                             *(dev(i) for i in (a, sa, None, w, sw, counts, offsets)), q, s)
    torch.cuda.synchronize()
    bad = torch.isnan(s).all(dim=1).cpu().numpy()
    assert bad[[3, 5]].all() and bad.sum() == 2


def test_transposed_weights_give_the_data_gradient():
    """dA = dY W through the same call on W transposed, against differences of
    the product itself (both linear: equal to rounding)."""
    T, E, k, K, N = 60, 3, 2, 256, 384
    rng = np.random.default_rng(13)
    a, sa, _, w, sw, counts, offsets = inputs(rng, T, E, k, K, N, False)
    dy, sdy = codes8(rng, (T * k, N)), scales(rng, (T * k, L.blocks(N)))
    wt, swt = np.ascontiguousarray(w.transpose(0, 2, 1)), np.ascontiguousarray(sw.transpose(0, 2, 1))
    da = f64(run_gemm(T, E, k, N, K, (dy, sdy, None, wt, swt, counts, offsets), B.MOE_BF16, B.MOE_FLAG_OUT_F32))
    y, mag = L.expert_gemm(a, sa, None, k, w, sw, counts, offsets, T * k)
    lhs = (y * L.values8(dy, sdy)).sum()
    rhs = (da * L.values8(a, sa)).sum()
    assert abs(lhs - rhs) <= (N + 8) * 2 * U * (mag * np.abs(L.values8(dy, sdy))).sum()


def test_bad_tables_stay_in_bounds():
    """Counts, offsets and src that no layout writes: an unspecified result,
    inside the buffers."""
    say("[case] product with corrupted tables")
    T, E, k, K, N = 200, 7, 2, 144, 72
    rng = np.random.default_rng(14)
    a, sa, src, w, sw, counts, offsets = inputs(rng, T, E, k, K, N, True)
    big = np.int32(2 ** 31 - 1)
    for name, c, o, s in (("huge counts", np.full(E, big), offsets, src), ("negative counts", -counts, offsets, src),
                          ("far offsets", counts, np.full(E, big), src),
                          ("negative offsets", counts, np.full(E, -big), src),
                          ("bad src", counts, offsets, np.where(np.arange(T * k) % 2, big, -big).astype(np.int32))):
        say(f"[case] {name}")
        run_gemm(T, E, k, K, N, (a, sa, s, w, sw, c.astype(np.int32), o.astype(np.int32)), B.MOE_BF16)
        q = torch.full((T * k + 2, N // 2 // 16 * 16), 7.0, device="cuda").to(B.E4M3)
        sc = torch.full((T * k + 2, 1), 7.0, device="cuda")
        I = q.shape[1]
        ww, sww = w[:, :2 * I], sw[:, :L.blocks(2 * I)]
        B.moe_expert_gemm_swiglu(B.make_problem(T, E, k, 8, 1, B.MOE_BF16), K, I,
                                 *(dev(i) for i in (a, sa, s, ww, sww, c.astype(np.int32), o.astype(np.int32))), q, sc)
        torch.cuda.synchronize()
        assert (q[T * k:].float() == 7.0).all() and (sc[T * k:] == 7.0).all()


def test_rows_past_four_gib():
    """Codes of 5 GiB: the last rows' offsets pass 32 bits."""
    T, K, N = 320000, 16384, 8
    say(f"[case] product T={T} K={K} N={N}")
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    a = torch.empty(T, K, dtype=torch.uint8, device="cuda")
    for part in a.split(20000):
        part.random_(0, 0x60, generator=g)
    rng = np.random.default_rng(15)
    sa, w, sw = scales(rng, (T, K // 128)), codes8(rng, (1, N, K)), scales(rng, (1, 1, K // 128), 1e-4)
    y = torch.empty(T, N, device="cuda")
    B.moe_expert_gemm(B.make_problem(T, 1, 1, 8, 1, B.MOE_BF16, B.MOE_FLAG_OUT_F32), K, N, a.view(B.E4M3), dev(sa),
                      None, dev(w), dev(sw), dev(np.array([T], np.int32)), dev(np.array([0], np.int32)), y)
    torch.cuda.synchronize()
    rows = np.array([0, 131071, 131072, 262143, 262144, T - 257, T - 1])
    av = a[torch.from_numpy(rows).cuda()].cpu().numpy()
    want, mag = L.expert_gemm(av, sa[rows], None, 1, w, sw, [len(rows)], [0], len(rows))
    assert_within(f64(y[torch.from_numpy(rows).cuda()]), want, (K + K // 128 + 4) * 2 * U * mag, "y")


@pytest.mark.parametrize("K,N", [(16, 16), (144, 272), (640, 512), (1424, 2096)])
def test_a_row_does_not_depend_on_its_neighbours(K, N):
    """The same rows in segments of 1 to 300: a segment of at most 16 takes
    other waves than a larger one, and tiles have 1 to 4 units."""
    say(f"[case] neighbours K={K} N={N}")
    rng = np.random.default_rng(K)
    T = 300
    a, sa, _, w, sw, _, _ = inputs(rng, T, 1, 1, K, N, False)
    zero = np.zeros(1, np.int32)
    I = N // 2 // 16 * 16

    def run(n):
        inp = (a[:n], sa[:n], None, w, sw, np.array([n], np.int32), zero)
        y = [run_gemm(n, 1, 1, K, N, inp, B.MOE_BF16), run_gemm(n, 1, 1, K, N, inp, B.MOE_F16, B.MOE_FLAG_OUT_F32)]
        if I == 0:
            return y
        q, s = torch.empty(n, I, device="cuda").to(B.E4M3), torch.empty(n, L.blocks(I), device="cuda")
        B.moe_expert_gemm_swiglu(B.make_problem(n, 1, 1, 8, 1, B.MOE_BF16), K, I,
                                 *(dev(i) for i in (a[:n], sa[:n], None, w[:, :2 * I], sw[:, :L.blocks(2 * I)],
                                                    inp[5], zero)), q, s)
        torch.cuda.synchronize()
        return y + [q, s]

    want = run(T)
    for n in (1, 3, 15, 16, 17, 33, 64, 65, 130, 250):
        for i, (x, y) in enumerate(zip(run(n), want)):
            assert torch.equal(x.view(torch.uint8), y[:n].contiguous().view(torch.uint8)), (n, i)


def test_product_repeats_bit_for_bit_on_two_streams():
    T, E, k, K, N = 300, 16, 4, 512, 256
    rng = np.random.default_rng(16)
    one = inputs(rng, T, E, k, K, N, True, "skewed")
    two = inputs(rng, T, E, k, K, N, True)
    want = [run_gemm(T, E, k, K, N, i, B.MOE_F16) for i in (one, two)]
    p = B.make_problem(T, E, k, 8, 1, B.MOE_F16)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    devs = [[dev(i) for i in inp] for inp in (one, two)]
    outs = [torch.zeros(T * k, N, dtype=torch.float16, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for st, d, o in zip(streams, devs, outs):
            B.moe_expert_gemm(p, K, N, *d, o, st)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o.view(torch.int16), w.view(torch.int16))


def test_half_a_step_of_the_output_is_reached():
    """The bound of a 16-bit output is its rounding: nothing else moves a sum
    of a few small integers."""
    T, E, k, K, N = 8, 1, 1, 16, 8
    a = np.zeros((T, K), np.uint8)
    a[:, 0], a[:, 1] = 0x78, 0x38          # 256 and 1
    w = np.zeros((1, N, K), np.uint8)
    w[0, :, 0], w[0, :, 1] = 0x38, 0x38
    one = np.ones((T, 1), np.float32)
    y = run_gemm(T, E, k, K, N, (a, one, None, w, np.ones((1, 1, 1), np.float32), np.array([T], np.int32),
                                 np.zeros(1, np.int32)), B.MOE_BF16)
    assert (y.float() == 256.0).all() and HALF[B.MOE_BF16] * 257 >= 1  # 257 to even


def exact_sum_bound(y, mag, K, act):
    """Exact products summed in fp32 (K + K / 128 + 4 truncations) and one
    rounding to the activation format."""
    d = (K + L.blocks(K) + 4) * 2 * U * mag
    return d + round_bound(np.abs(y) + d, act)


def with_outliers(K, rng, T, N):
    """Codes of one large value beside seven small ones of one sign in every
    group of eight, the small ones' products below 2^-13 of the large one's; in
    every second row normal codes with one column in 128 at the format's end."""
    a = np.full((T, K), 0x0f, np.uint8)           # 15 2^-9
    a[:, ::8] = 0x78                              # 256
    a[1::2] = codes8(rng, (T // 2, K)) & 0x9f     # at most 2^-3
    a[1::2, ::128] = 0x7e                         # 448
    return a, np.full((1, N, K), 0x38, np.uint8)  # 1


@pytest.mark.parametrize("T", [4, 40, 150, 300])
@pytest.mark.parametrize("K", [16, 256, 400, 1024])
def test_fp16_sums_are_exact_beside_outliers(T, K):
    """An fp16 row's only rounding beside fp32's is its own: with products cut
    off below the largest of eight, the sum of 256 + 7 15 2^-9 a group came out
    1.6 half steps low."""
    say(f"[case] product with outliers T={T} K={K}")
    rng, N, act = np.random.default_rng(T + K), 136, B.MOE_F16
    a, w = with_outliers(K, rng, T, N)
    one, seg = np.ones((T, L.blocks(K)), np.float32), (np.array([T], np.int32), np.zeros(1, np.int32))
    inp = (a, one, None, w, np.ones((1, 2, L.blocks(K)), np.float32), *seg)
    y, mag = L.expert_gemm(*inp[:3], 1, *inp[3:], T)
    assert np.abs(y).max() < 65504
    got = f64(run_gemm(T, 1, 1, K, N, inp, act))
    print("worst error in half steps:", (np.abs(got - y) / (HALF[act] * np.abs(y))).max(), flush=True)
    assert_within(got, y, exact_sum_bound(y, mag, K, act), "y")


@pytest.mark.parametrize("T", [4, 40, 150, 300])
@pytest.mark.parametrize("K", [16, 256, 400, 1024])
def test_bf16_sums_beside_outliers(T, K):
    """In bf16 the cut-off leaves at most 7 2^-13 of each group's largest
    product, 0.22 of half a step of a sum of one sign."""
    say(f"[case] product with outliers in bf16 T={T} K={K}")
    rng, N, act = np.random.default_rng(T + K), 136, B.MOE_BF16
    a, w = with_outliers(K, rng, T, N)
    one, seg = np.ones((T, L.blocks(K)), np.float32), (np.array([T], np.int32), np.zeros(1, np.int32))
    inp = (a, one, None, w, np.ones((1, 2, L.blocks(K)), np.float32), *seg)
    y, mag = L.expert_gemm(*inp[:3], 1, *inp[3:], T)
    got = f64(run_gemm(T, 1, 1, K, N, inp, act))
    print("worst error in half steps:", (np.abs(got - y) / (HALF[act] * np.abs(y))).max(), flush=True)
    lost = 7 / 8 * lost_in_groups(inp, 1, T, N)
    assert_within(got, y, exact_sum_bound(y, mag, K, act) + lost * (1 + HALF[act]), "y")


@pytest.mark.parametrize("T", [1, 40, 200])
def test_fp16_rows_are_the_fp32_rows_rounded(T):
    """The same sums under either output format, bit for bit."""
    say(f"[case] exact sums in two formats T={T}")
    E, k, K, N = 3, 2, 272, 520
    inp = inputs(np.random.default_rng(T), T, E, k, K, N, True)
    f32 = run_gemm(T, E, k, K, N, inp, B.MOE_BF16, B.MOE_FLAG_OUT_F32)
    assert torch.equal(run_gemm(T, E, k, K, N, inp, B.MOE_F16).view(torch.int16), f32.half().view(torch.int16))


@pytest.mark.parametrize("T", [4, 40, 150, 300])
@pytest.mark.parametrize("K", [16, 256, 400, 1024])
def test_bf16_sums_are_exact_when_asked_for(T, K):
    """With MOE_FLAG_EXACT_SUMS nothing is cut off beside outliers, also where
    the large products cancel and the small ones are the sum."""
    say(f"[case] exact sums in bf16 T={T} K={K}")
    rng, N, act = np.random.default_rng(T + K), 136, B.MOE_BF16
    a, w = with_outliers(K, rng, T, N)
    a[2::4, 8::16] |= 0x80  # the large ones of every second group: their sum is 0
    a[2::4, :16] = 0x0f
    a[2::4, 0], a[2::4, 8] = 0x78, 0xf8
    if K % 32 == 16:
        a[2::4, K - 16:] = 0x0f
    one, seg = np.ones((T, L.blocks(K)), np.float32), (np.array([T], np.int32), np.zeros(1, np.int32))
    inp = (a, one, None, w, np.ones((1, 2, L.blocks(K)), np.float32), *seg)
    y, mag = L.expert_gemm(*inp[:3], 1, *inp[3:], T)
    out = torch.full((T + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
    B.moe_expert_gemm(B.make_problem(T, 1, 1, 8, 1, act, B.MOE_FLAG_EXACT_SUMS), K, N, *(dev(i) for i in inp), out)
    torch.cuda.synchronize()
    assert (out[T:] == 7.0).all()
    assert_within(f64(out[:T]), y, exact_sum_bound(y, mag, K, act), "y")


@pytest.mark.parametrize("T", [1, 40, 200])
def test_exact_bf16_rows_are_the_fp32_rows_rounded(T):
    say(f"[case] exact sums in bf16 and fp32 T={T}")
    E, k, K, N = 3, 2, 272, 520
    for gather in (True, False):
        inp = inputs(np.random.default_rng(T), T, E, k, K, N, gather)
        f32 = run_gemm(T, E, k, K, N, inp, B.MOE_BF16, B.MOE_FLAG_OUT_F32)
        both = run_gemm(T, E, k, K, N, inp, B.MOE_BF16, B.MOE_FLAG_OUT_F32 | B.MOE_FLAG_EXACT_SUMS)
        assert torch.equal(both, f32)
        out = torch.empty(T * k, N, dtype=torch.bfloat16, device="cuda")
        B.moe_expert_gemm(B.make_problem(T, E, k, 8, 1, B.MOE_BF16, B.MOE_FLAG_EXACT_SUMS), K, N,
                          *(dev(i) for i in inp), out)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), f32.bfloat16().view(torch.int16))


@pytest.mark.parametrize("T", [3, 100])
def test_scales_whose_product_is_just_finite(T):
    """Row scales of 2^70 by weight scales of 2^57: blocks of zeros are zeros,
    and small codes what they stand for."""
    say(f"[case] scales near the end of fp32 T={T}")
    K, N = 400, 72
    a, w = np.zeros((T, K), np.uint8), np.full((1, N, K), 0x01, np.uint8)  # 2^-9
    a[1:, 130], a[2:, 399] = 0x01, 0x81  # 2^-9, -2^-9
    sa, sw = np.full((T, 4), 2.0 ** 70, np.float32), np.full((1, 1, 4), 2.0 ** 57, np.float32)
    inp = (a, sa, None, w, sw, np.array([T], np.int32), np.zeros(1, np.int32))
    want = np.zeros((T, 1))
    want[1] = 2.0 ** 109
    for act, flags in ((B.MOE_BF16, 0), (B.MOE_BF16, B.MOE_FLAG_OUT_F32)):
        assert (f64(run_gemm(T, 1, 1, K, N, inp, act, flags)) == want).all(), flags
    q, s = torch.empty(T, 32, device="cuda").to(B.E4M3), torch.empty(T, 1, device="cuda")
    B.moe_expert_gemm_swiglu(B.make_problem(T, 1, 1, 8, 1, B.MOE_BF16), K, 32,
                             *(dev(i) for i in (a, sa, None, w[:, :64], sw, inp[5], inp[6])), q, s)
    torch.cuda.synchronize()
    rest = [0] + list(range(2, T))
    assert (q[rest].float() == 0).all() and (s[rest] == np.float32(2.0 ** -100) / np.float32(448)).all()


def test_largest_row_scale_by_a_weight_scale_of_256():
    """What the header says of the rows this library writes: the largest scale
    there is, of a row of FLT_MAX, by 256 is finite."""
    say("[case] largest row scale")
    T, K, N = 5, 128, 16
    far = np.float32(np.finfo(np.float32).max)
    # a row of FLT_MAX out of the SwiGLU: silu(FLT_MAX) * 1
    a, w = np.zeros((T, 16), np.uint8), np.zeros((1, 2 * K, 16), np.uint8)
    a[:, 0], a[:, 1], w[0, :K, 0], w[0, K:, 1] = 0x38, 0x38, 0x38, 0x38
    one, seg = np.ones((T, 1), np.float32), (np.array([T], np.int32), np.zeros(1, np.int32))
    q, s = torch.empty(T, K, device="cuda").to(B.E4M3), torch.empty(T, 1, device="cuda")
    B.moe_expert_gemm_swiglu(B.make_problem(T, 1, 1, 8, 1, B.MOE_BF16), 16, K,
                             *(dev(i) for i in (a, one, None, w, np.array([far, 1.0], np.float32).reshape(1, 2, 1),
                                                *seg)), q, s)
    torch.cuda.synchronize()
    assert (q.float() == 448).all() and torch.isfinite(s).all()
    assert (np.abs(f64(s) * 448 / float(far) - 1) <= 2 * U).all()
    # rows of that scale with codes of 0 and of 1, by weights of 2^-9 in a block of scale 256
    zero = np.zeros((T, K), np.uint8)
    wv = np.zeros((1, N, K), np.uint8)
    wv[0, :, 5] = 0x01
    sw = np.full((1, 1, 1), 256.0, np.float32)
    for flags in (0, B.MOE_FLAG_OUT_F32):
        got = f64(run_gemm(T, 1, 1, K, N, (zero, s.cpu().numpy(), None, wv, sw, *seg), B.MOE_BF16, flags))
        assert (got == 0).all()
        one_code = np.full((T, K), 0x38, np.uint8)
        got = f64(run_gemm(T, 1, 1, K, N, (one_code, s.cpu().numpy(), None, wv, sw, *seg), B.MOE_BF16, flags))
        want = np.broadcast_to(f64(s) * 0.5, got.shape)  # 256 2^-9
        assert_within(got, want, (U + HALF[B.MOE_BF16]) * want, "y")


@pytest.mark.parametrize("flags", [0, B.MOE_FLAG_OUT_F32])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T", [3, 90])
def test_small_products_beside_large_ones_count(T, act, flags):
    """Sums whose rounded value changes if any of their products is lost:
    256 + 1 + 1 and 256 + 3 (258 and 260 in bf16, as they are in fp16 and fp32),
    256 + 1 (exact in fp16 and fp32), 256 + 2 - 1 + 1."""
    say(f"[case] small integers T={T} act={act} flags={flags}")
    K, N = 32, 8
    rows = [[(0x78, 1), (0x38, 1), (0x38, 1)], [(0x78, 1), (0x44, 1)], [(0x78, 1), (0x38, 1)],
            [(0x78, 1), (0x40, 1), (0x38, -1), (0x38, 1)]]
    want = np.array([258.0, 259.0, 257.0, 258.0])
    if act == B.MOE_BF16 and not flags:
        want = np.array([258.0, 260.0, 256.0, 258.0])  # 259 and 257 to even
    one = np.ones((T, 1), np.float32)
    for first in (0, 7, 15):  # of the places: one group of eight, two, two chunks
        a, w = np.zeros((T, K), np.uint8), np.zeros((1, N, K), np.uint8)
        w[0] = 0x38
        for r in range(T):
            for j, (c, sign) in enumerate(rows[r % 4]):
                a[r, first + j] = c | (0x80 if sign < 0 else 0)
        y = run_gemm(T, 1, 1, K, N, (a, one, None, w, np.ones((1, 1, 1), np.float32), np.array([T], np.int32),
                                     np.zeros(1, np.int32)), act, flags)
        assert (f64(y) == want[np.arange(T) % 4][:, None]).all(), first
