"""The gradient of the experts' weights on the GPU against the oracle, and the
training of a layer's down weights from the combine's gradient to AdamW's step.

A sum of n rows is off by at most (n + 24) 2 u of its terms' magnitudes (a matrix
instruction's additions may truncate; shares of the rows are added up), then one
rounding; with `add` one more addition."""
import numpy as np
import pytest
import torch

import oracle
from combine_router_topk_amd import binding as B
from combine_router_topk_amd import path as P
from layercheck import ACTS, HALF, U, assert_within, bits16, dev, f64, round_bound
from oracle import train
from pathcheck import say
from test_packed_gemm_gpu import segments_of

pytestmark = pytest.mark.gpu


def grad(p, K, N, a, src, dy, counts, offsets, add, dw, stream=None):
    ws = torch.full((B.moe_expert_weight_grad_workspace_bytes(p, K, N),), 255, dtype=torch.uint8, device="cuda")
    B.moe_expert_weight_grad(p, K, N, a, src, dy, counts, offsets, add, dw, ws, stream)


def check_grad(counts, k, K, N, act, gather, out="16", seed=0):
    counts = np.asarray(counts, np.int32)
    say(f"[case] weight grad counts={counts[:6]}.. k={k} K={K} N={N} act={act} gather={gather} out={out}")
    rng = np.random.default_rng(seed + K + N + counts.size)
    E = counts.size
    T, src, offsets = segments_of(rng, counts, k)
    p = B.make_problem(T, E, k, 8, 1, act, 0 if out == "16" else B.MOE_FLAG_OUT_F32)
    a, dy = bits16(rng, (T if gather else T * k, K), act), bits16(rng, (T * k, N), act, 0.1)
    old = rng.standard_normal((E, N, K)).astype(np.float32)
    whole = torch.full((E * N * K + 64,), -7.0, dtype=torch.float32 if out != "16" else dev(a, act).dtype, device="cuda")
    dw = whole[:E * N * K].view(E, N, K)
    if out == "add":
        dw.copy_(torch.from_numpy(old))
    args = dev(a, act), dev(src) if gather else None, dev(dy, act), dev(counts), dev(offsets)
    grad(p, K, N, *args, out == "add", dw)
    torch.cuda.synchronize()
    assert (whole[E * N * K:] == -7).all()
    val = lambda b: oracle.decode16(b, act).astype(np.float64)  # noqa: E731
    want, mag = train.weight_grad(val(dy), val(a), src if gather else None, k, counts, offsets, E)
    bound = (counts[:, None, None] + 24) * 2 * U * mag
    if out == "add":
        bound = bound + U * (np.abs(old + want) + bound)
        want = want + old
    elif out == "16":
        bound = bound + round_bound(np.abs(want) + bound, act)
    else:
        bound = bound + 1e-30
    assert_within(f64(dw), want, bound, "dw")
    assert not f64(dw)[counts == 0].any() or out == "add"
    return dw, args, p


CASES = [([1], 1, 8, 8), ([3, 0, 5], 2, 128, 16), ([0, 0, 7, 1], 1, 136, 40), ([32, 33, 31, 64, 0, 2], 3, 264, 72),
         ([200], 1, 256, 256), ([129, 0, 64, 1, 300], 2, 264, 520), ([5] * 30, 2, 96, 24), ([1000, 2], 2, 512, 264),
         ([0, 0], 1, 16, 24)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("out", ["16", "f32", "add"])
@pytest.mark.parametrize("counts,k,K,N", CASES)
def test_weight_grad(counts, k, K, N, act, out):
    check_grad(counts, k, K, N, act, gather=k > 1, out=out)


def test_rows_in_shares():
    """Few tiles and many rows: the rows are split and the shares added up."""
    for counts, k, K, N in (([4000, 96], 1, 256, 264), ([3000, 1, 999, 4000], 2, 40, 64), ([2048], 1, 8, 8)):
        n = sum(counts)
        p = B.make_problem(n // k, len(counts), k, 8, 1, B.MOE_BF16)
        assert B.moe_expert_weight_grad_workspace_bytes(p, K, N) >= 2 * len(counts) * N * K * 4
        for out in ("16", "f32", "add"):
            check_grad(counts, k, K, N, B.MOE_BF16, k > 1, out)
    check_grad([50, 5000], 1, 48, 24, B.MOE_F16, False, "add")


@pytest.mark.parametrize("out", ["16", "f32", "add"])
def test_skewed_rows_are_cut(out):
    """One expert with most of the rows beside experts with few and none, in order and
    in reverse, at more tiles than one."""
    counts = [0, 5, 3000, 40, 0, 700, 1, 350]
    for c in (counts, counts[::-1]):
        check_grad(c, 4, 520, 136, B.MOE_F16, True, out)
    check_grad([9000] + [10] * 100, 2, 264, 264, B.MOE_BF16, False, out)


def test_plans_of_overlapping_segments_stay_inside():
    """Counts that add up to many times the rows: every expert has all of them."""
    say("[case] weight grad, overlapping segments")
    T, E, N, K = 4096, 64, 24, 16
    p = B.make_problem(T, E, 1, 8, 1, B.MOE_BF16, B.MOE_FLAG_OUT_F32)
    a, dy = torch.ones(T, K, dtype=torch.bfloat16, device="cuda"), torch.ones(T, N, dtype=torch.bfloat16, device="cuda")
    counts, offsets = torch.full((E,), T, dtype=torch.int32, device="cuda"), torch.zeros(E, dtype=torch.int32, device="cuda")
    need = B.moe_expert_weight_grad_workspace_bytes(p, K, N)
    assert need > 0
    ws = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    dw = torch.empty(E, N, K, device="cuda")
    B.moe_expert_weight_grad(p, K, N, a, None, dy, counts, offsets, False, dw, ws)
    torch.cuda.synchronize()
    assert (dw == T).all() and (ws[need:] == 77).all()


@pytest.mark.parametrize("E,k,K,N,counts,act,out", [
    (1024, 2, 520, 264, [0, 1, 33, 64, 65, 100, 7, 32], B.MOE_BF16, "add"),
    (1024, 1, 776, 264, [0, 40, 1100, 0, 0, 96, 0, 0], B.MOE_F16, "16"),
    (16, 2, 4096, 4096, [0, 1, 33, 64, 65, 100, 1090, 33], B.MOE_BF16, "16"),
    (16, 2, 4104, 4096, [70, 35, 64, 65], B.MOE_F16, "f32")])
def test_thousands_of_tiles(E, k, K, N, counts, act, out):
    """Rows of no step, one, two and more, and more than have their sources in LDS."""
    say(f"[case] weight grad of many tiles E={E} K={K} N={N} {out}")
    rng = np.random.default_rng(K)
    counts = np.asarray(counts * (E // len(counts)), np.int32)
    T, src, offsets = segments_of(rng, counts, k)
    p = B.make_problem(T, E, k, 8, 1, act, 0 if out == "16" else B.MOE_FLAG_OUT_F32)
    torch.manual_seed(K)
    dt = torch.float16 if act == B.MOE_F16 else torch.bfloat16
    a, dy = torch.randn(T, K, device="cuda").to(dt), torch.randn(T * k, N, device="cuda").to(dt)
    dw = torch.full((E, N, K), 0.5, dtype=dt if out == "16" else torch.float32, device="cuda")
    grad(p, K, N, a, dev(src), dy, dev(counts), dev(offsets), out == "add", dw)
    torch.cuda.synchronize()
    rows = torch.from_numpy(src // k).cuda().long()
    for e in range(E) if E < 100 else [*range(16), *range(500, 508), *range(E - 8, E)]:
        r = slice(int(offsets[e]), int(offsets[e] + counts[e]))
        av, dv = a[rows[r]].double(), dy[r].double()
        want, size = dv.T @ av, dv.abs().T @ av.abs()
        bound = (int(counts[e]) + 24) * 2 * U * size
        if out == "add":
            want = want + 0.5
            bound = bound + U * want.abs() * 1.01
        elif out == "16":
            bound = bound + HALF[act] * (want.abs() + bound) * 1.01 + 2.0 ** -25
        assert ((dw[e].double() - want).abs() <= bound + 1e-30).all(), e


def test_many_experts():
    check_grad([4] * 1024, 2, 40, 16, B.MOE_BF16, True, "f32")
    check_grad([0] * 500 + [70] * 20 + [0] * 400, 2, 72, 264, B.MOE_F16, False, "16")


def test_no_rows():
    for add in (False, True):
        p = B.make_problem(0, 3, 1, 8, 1, B.MOE_F16, B.MOE_FLAG_OUT_F32)
        dw = torch.full((3, 16, 24), 5.0, device="cuda")
        z = torch.zeros(3, dtype=torch.int32, device="cuda")
        B.moe_expert_weight_grad(p, 24, 16, None, None, None, z, z, add, dw, None)
        torch.cuda.synchronize()
        assert (dw == (5.0 if add else 0.0)).all()


@pytest.mark.parametrize("counts", [[5, 8, 3], [700, 100, 40]])
def test_non_finite_rows_stay_in_their_expert_and_column(counts):
    rng = np.random.default_rng(1)
    counts = np.asarray(counts, np.int32)
    n, K, N, act = int(counts.sum()), 264, 72, B.MOE_BF16
    T, src, offsets = segments_of(rng, counts, 1)
    p = B.make_problem(n, 3, 1, 8, 1, act, B.MOE_FLAG_OUT_F32)
    a, dy = bits16(rng, (n, K), act), bits16(rng, (n, N), act)
    out = []
    for bad in (False, True):
        aa, dd = a.copy(), dy.copy()
        if bad:
            aa[2, 7], dd[counts[0] + 1, 9] = 0x7fc0, 0x7f80
        dw = torch.empty(3, N, K, device="cuda")
        grad(p, K, N, dev(aa, act), None, dev(dd, act), dev(counts), dev(offsets), False, dw)
        torch.cuda.synchronize()
        out.append(f64(dw))
    good, got = out
    assert np.isnan(got[0, :, 7]).all() and not np.isfinite(got[1, 9, :]).any()
    keep = np.ones_like(good, bool)
    keep[0, :, 7], keep[1, 9, :] = False, False
    assert np.array_equal(got[keep], good[keep])


def test_bad_tables_stay_inside():
    say("[case] weight grad with bad tables")
    for T in (8, 3000):
        p = B.make_problem(T, 3, 1, 8, 1, B.MOE_F16, B.MOE_FLAG_OUT_F32)
        a, dy = (torch.ones(T, 24, dtype=torch.float16, device="cuda") for _ in range(2))
        src = torch.full((T,), 1 << 30, dtype=torch.int32, device="cuda")
        src[0] = -5
        counts = torch.tensor([1 << 30, -3, 5], dtype=torch.int32, device="cuda")
        offsets = torch.tensor([-4, 2, T - 1], dtype=torch.int32, device="cuda")
        dw = torch.empty(3, 24, 24, device="cuda")
        grad(p, 24, 24, a, src, dy, counts, offsets, False, dw)
        torch.cuda.synchronize()
        assert (dw[0] == T).all() and (dw[1] == 0).all() and (dw[2] == 1).all()


def test_repeats_streams_and_graph():
    dw, args, p = check_grad([700, 300, 24], 2, 264, 136, B.MOE_BF16, True, "f32")
    want = dw.clone()
    side = torch.cuda.Stream()
    second = torch.empty_like(want)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        grad(p, 264, 136, *args, False, second)
    side.synchronize()
    assert torch.equal(second, want)
    ws = torch.empty(B.moe_expert_weight_grad_workspace_bytes(p, 264, 136), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_expert_weight_grad(p, 264, 136, *args, False, second, ws)
    for _ in range(3):
        second.fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(second, want)


def test_past_four_gigabytes():
    """Weights past 2^32 values and rows past 2^31: the last expert's and rows."""
    say("[case] weight grad, 40 experts of 8192 x 16384")
    E, N, K, act = 40, 8192, 16384, B.MOE_BF16
    rows = 140000
    a, dy = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda"), torch.zeros(rows, N, dtype=torch.bfloat16, device="cuda")
    torch.manual_seed(2)
    a[-3:], dy[-3:] = torch.randn(3, K, device="cuda").bfloat16(), torch.randn(3, N, device="cuda").bfloat16()
    counts, offsets = (torch.zeros(E, dtype=torch.int32, device="cuda") for _ in range(2))
    counts[E - 1], offsets[E - 1] = 200, rows - 200
    dw = torch.full((E, N, K), 9.0, dtype=torch.bfloat16, device="cuda")
    p = B.make_problem(rows, E, 1, 8, 1, act)
    grad(p, K, N, a, None, dy, counts, offsets, False, dw)
    torch.cuda.synchronize()
    want = dy[-3:, -100:].double().T @ a[-3:, -300:].double()
    size = dy[-3:, -100:].double().abs().T @ a[-3:, -300:].double().abs()
    got = dw[E - 1, -100:, -300:].double()
    assert ((got - want).abs() <= HALF[act] * want.abs() * 1.01 + 60 * U * size).all()
    assert not dw[:E - 1].any() and bool(dw[E - 1, :, -1].any())


def test_gradients_against_differences():
    """The loss sum(out * r) of a layer y = W_e x with its combine: the gradient
    along a direction against a central difference of the loss in fp64."""
    rng = np.random.default_rng(8)
    T, E, k, K, N, act = 40, 4, 2, 48, 32, B.MOE_F16
    counts = np.bincount(rng.integers(0, E, T * k), minlength=E)
    _, src, offsets = segments_of(rng, counts, k)
    a, dy = bits16(rng, (T, K), act), bits16(rng, (T * k, N), act, 0.1)
    p = B.make_problem(T, E, k, 8, 1, act, B.MOE_FLAG_OUT_F32)
    dw = torch.empty(E, N, K, device="cuda")
    grad(p, K, N, dev(a, act), dev(src), dev(dy, act), dev(counts.astype(np.int32)), dev(offsets), False, dw)
    torch.cuda.synchronize()
    av, dv = oracle.decode16(a, act).astype(np.float64), oracle.decode16(dy, act).astype(np.float64)
    way = rng.standard_normal((E, N, K))
    expert = np.repeat(np.arange(E), counts)
    loss = lambda w: sum(float(dv[r] @ (w[expert[r]] @ av[src[r] // k])) for r in range(T * k))  # noqa: E731
    w = rng.standard_normal((E, N, K))
    slope = (loss(w + way) - loss(w - way)) / 2
    got = float((f64(dw) * way).sum())
    size = sum(float(np.abs(dv[r]) @ (np.abs(way[expert[r]]) @ np.abs(av[src[r] // k]))) for r in range(T * k))
    assert abs(got - slope) <= 2 * U * (counts.max() + 24) * size + 1e-12 * abs(loss(w))


def test_a_training_step_and_the_weights_it_serves():
    """Routing, the combine's gradient, the down weights' gradient, an AdamW step
    and the new weights in 4 bits: each beside torch's fp64 result from the step
    before, and the loss's gradient beside autograd's."""
    say("[case] a training step")
    T, E, k, H, I, act = 64, 8, 2, 128, 64, B.MOE_BF16
    torch.manual_seed(3)
    p = B.make_problem(T, E, k, H, 1, act)
    b = P.allocate(p, torch.randn(T, E), torch.randn(T, H).bfloat16())
    P.route_assign_layout(b)
    inner = torch.randn(T * k, I, device="cuda").bfloat16()
    w = (torch.randn(E, H, I, device="cuda") / I ** 0.5).bfloat16()
    expert = b.idx.long()[b.src.long()]
    b.y.copy_(torch.bmm(w[expert].float(), inner.float()[:, :, None])[:, :, 0])
    P.combine(b)
    dout = torch.randn(T, H, device="cuda").bfloat16()
    dy, dgate = torch.empty_like(b.y), torch.empty(T * k, device="cuda")
    B.moe_combine_backward(p, dout, b.y, b.pos, b.w, dy, dgate)
    tr = P.allocate_weight_grad(b, H, I)
    P.expert_weight_grad(b, tr, inner, None, dy)
    torch.cuda.synchronize()
    w64 = w.double().requires_grad_()
    y = torch.bmm(w64[expert], inner.double()[:, :, None])[:, :, 0]
    out = (b.w.double().view(T, k)[:, :, None] * y[b.pos.long()].view(T, k, H)).sum(1)
    out.backward(dout.double())
    size = torch.zeros(E, H, I, dtype=torch.float64, device="cuda")
    size.index_add_(0, expert, dy.double().abs()[:, :, None] * inner.double().abs()[:, None, :])
    # dy was rounded to bf16, and sums of at most 128 rows are in fp32
    assert ((tr.dw.double() - w64.grad).abs() <= size * (HALF[act] * 1.02 + 2 * U * 160)).all()

    master = w.float()
    state = {key: torch.zeros(E, H, I, device="cuda") for key in ("m", "v")}
    plan = B.AdamWTensors([dict(w=w, master=master, g=tr.dw, weight_decay=0.1, **state)])
    before = master.double().clone()
    B.moe_adamw_step(B.make_adamw(1e-2, 0.9, 0.999, 1e-8, 1), plan)
    torch.cuda.synchronize()
    g = tr.dw.double()
    want = before - 1e-2 * 0.1 * before - 1e-2 * g / (g.abs() + 1e-8)
    assert ((master.double() - want).abs() <= 32 * U * 1e-2 + 3 * U * before.abs()).all()
    assert torch.equal(w, master.bfloat16())

    f = B.make_packed_format(B.MOE_PACKED_E2M1, 32, act)
    packed = P.pack_weights(master, f)
    back = P.unpack_weights(packed, H, I, f)
    y4 = torch.empty_like(b.y)
    B.moe_expert_gemm_packed(p, f, I, H, inner, None, packed, b.counts, b.expert_offsets, y4)
    torch.cuda.synchronize()
    ref = torch.bmm(back[expert].double(), inner.double()[:, :, None])[:, :, 0]
    size = torch.bmm(back[expert].double().abs(), inner.double().abs()[:, :, None])[:, :, 0]
    assert ((y4.double() - ref).abs() <= HALF[act] * ref.abs() * 1.01 + 2 * U * (I + 16) * size).all()
