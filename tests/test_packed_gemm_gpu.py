"""The experts' products with 4-bit weights on the GPU against the oracle.

Bounds as in test_packed_layer_gpu: a sum of K terms is off by at most (K + K /
32 + 8) 2 u of the magnitudes of what is summed, then one rounding."""
import numpy as np
import pytest
import torch

import oracle
from combine_router_topk_amd import binding as B
from layercheck import ACTS, U, assert_within, bits16, dev, f64, round_bound
from oracle import layer as L
from oracle import packed as O
from packedcheck import FORMATS, Weights
from pathcheck import say
from test_packed_layer_gpu import inner_bounds

pytestmark = pytest.mark.gpu


def segments_of(rng, counts, k):
    """(T, src, offsets) of a batch whose experts take `counts` rows, sum a
    multiple of k: the pairs in random order, sorted by expert."""
    n = int(sum(counts))
    assert n % k == 0
    offsets = np.cumsum(counts) - counts
    src = np.concatenate([np.sort(part) for part in np.split(rng.permutation(n), offsets[1:])]) if n else np.zeros(0)
    return n // k, src.astype(np.int32), offsets.astype(np.int32)


def check_gemm(counts, k, K, N, act, codes, group, gather, swiglu=False, flags=0, seed=0, scale_act=None, w=None):
    """N: weight rows of the plain product, or I."""
    counts = np.asarray(counts, np.int32)
    say(f"[case] packed product counts={counts[:6]}.. k={k} K={K} N={N} act={act} codes={codes} group={group} "
        f"gather={gather} swiglu={swiglu} flags={flags}")
    rng = np.random.default_rng(seed + K + N + counts.size)
    E = counts.size
    T, src, offsets = segments_of(rng, counts, k)
    p = B.make_problem(T, E, k, 8, 1, act, flags)
    a = bits16(rng, (T if gather else T * k, K), act)
    w = w or Weights(rng, E, 2 * N if swiglu else N, K, codes, group, scale_act or act)
    out_dt = torch.float32 if flags & B.MOE_FLAG_OUT_F32 and not swiglu else dev(a, act).dtype
    y = torch.full((T * k + 1, N), -7.0, dtype=out_dt, device="cuda")
    args = (dev(a, act), dev(src) if gather else None, w.dev, dev(counts), dev(offsets), y)
    if swiglu:
        B.moe_expert_gemm_swiglu_packed(p, w.format, K, N, *args)
    else:
        B.moe_expert_gemm_packed(p, w.format, K, N, *args)
    torch.cuda.synchronize()
    got = f64(y)
    assert (got[T * k] == -7).all()
    av = oracle.decode16(a, act).astype(np.float64)
    for e, r in L.segments(counts, offsets, T * k):
        rows = av[src[r] // k] if gather else av[r]
        v, mag = w.both(e)
        z, dz = rows @ v.T, (K + K / 32 + 8) * 2 * U * (np.abs(rows) @ mag.T)
        if swiglu:
            z, dz = inner_bounds(z, dz, N)
        if out_dt == torch.float32:
            assert_within(got[r], z, dz + 1e-30, f"y of expert {e}")
        else:
            assert_within(got[r], z, dz + round_bound(np.abs(z) + dz, act), f"y of expert {e}")
    return y[:T * k]


FEW = [([1], 1, 8, 8), ([3, 0, 5], 2, 128, 16), ([0, 0, 7, 1], 1, 136, 40), ([16, 17, 1, 0, 30, 2], 3, 264, 72),
       ([5] * 30, 2, 96, 24)]
MANY = [([200], 1, 128, 256), ([129, 0, 64, 1, 300], 2, 264, 72), ([128, 127, 65], 1, 40, 520), ([1000, 3, 1], 2, 512, 264),
        ([63] * 9, 3, 392, 136)]


@pytest.mark.parametrize("codes,group", FORMATS)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("counts,k,K,N", FEW + MANY)
def test_product(counts, k, K, N, act, codes, group):
    check_gemm(counts, k, K, N, act, codes, group, gather=k > 1)


@pytest.mark.parametrize("codes,group", FORMATS)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("counts,k,K,I", [([1], 1, 8, 16), ([3, 0, 5], 2, 128, 16), ([16, 17, 1, 0, 30, 2], 3, 264, 48),
                                          ([200], 1, 128, 128), ([129, 0, 64, 1, 300], 2, 264, 144), ([63] * 9, 3, 392, 272)])
def test_swiglu(counts, k, K, I, act, codes, group):
    check_gemm(counts, k, K, I, act, codes, group, gather=True, swiglu=True)


@pytest.mark.parametrize("codes,group", FORMATS)
def test_fp32_rows_and_scales_of_the_other_format(codes, group):
    for counts in ([5, 9, 2], [150, 0, 90]):
        for act in ACTS:
            check_gemm(counts, 2, 200, 72, act, codes, group, False, flags=B.MOE_FLAG_OUT_F32, scale_act=3 - act)


# Enough rows and weights for the kernel of many rows; its tiles have 128 rows (two halves)
# and 256 weight rows.
LARGE = [129, 0, 64, 1, 300, 65, 127, 128] * 3


def few_rows(rows, E, K, n):
    """The library's choice between its two kernels (its thin one if true)."""
    experts = min(rows, E)
    average = rows / experts
    thin = (rows / 16 + experts / 2) * n * K / 8.5e6
    tiles = np.ceil(experts * (1 if average <= 128 else average / 128 + 0.5) * -(-n // 256) / 256)
    return thin <= 5 + tiles * -(-K // 128) * (1.55 if average <= 48 else 2.2)


@pytest.mark.parametrize("codes,group", FORMATS)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("K,N,swiglu", [(264, 4104, False), (392, 4112, False), (264, 2064, True)])
def test_many_rows(K, N, swiglu, act, codes, group):
    assert not few_rows(sum(LARGE), len(LARGE), K, 2 * N if swiglu else N)
    check_gemm(LARGE, 2, K, N, act, codes, group, gather=True, swiglu=swiglu)


def test_many_rows_fp32_in_send_order_and_one_step():
    for codes, group in FORMATS[::2]:
        check_gemm(LARGE, 1, 264, 4104, B.MOE_F16, codes, group, False, flags=B.MOE_FLAG_OUT_F32, scale_act=B.MOE_BF16)
    counts = [40] * 300
    assert not few_rows(12000, 300, 128, 2056) and not few_rows(12000, 300, 104, 2056)
    check_gemm(counts, 2, 128, 2056, B.MOE_BF16, O.E2M1, 64, True)
    check_gemm(counts, 3, 104, 2056, B.MOE_BF16, O.INT, 32, True)


def test_many_rows_are_their_own_repeat_and_replay():
    rng = np.random.default_rng(1)
    counts = np.asarray(LARGE, np.int32)
    n, K, N, act, E = int(counts.sum()), 264, 4104, B.MOE_BF16, len(LARGE)
    offsets = (np.cumsum(counts) - counts).astype(np.int32)
    p = B.make_problem(n, E, 1, 8, 1, act)
    a = bits16(rng, (n, K), act)
    w = Weights(rng, E, N, K, O.INT, 64, act)

    def run(a, counts, stream=None):
        y = torch.full((n, N), -7.0, dtype=torch.bfloat16, device="cuda")
        args = dev(a, act), None, w.dev, dev(counts), dev(offsets), y
        torch.cuda.synchronize()
        B.moe_expert_gemm_packed(p, w.format, K, N, *args, stream)
        torch.cuda.synchronize()
        return y

    want = run(a, counts)
    bad = a.copy()
    bad[2, K - 1], bad[600, 3] = 0x7fc0, 0x7f80
    got = run(bad, counts, torch.cuda.Stream())
    rest = [r for r in range(n) if r not in (2, 600)]
    assert torch.equal(got[rest], want[rest]) and torch.isnan(got[2]).all() and not torch.isfinite(got[600]).any()
    fewer = counts.copy()
    fewer[0] -= 70
    got = run(a, fewer)
    gap = list(range(int(counts[0]) - 70, int(counts[0])))
    rest = [r for r in range(n) if r not in gap]
    assert torch.equal(got[rest], want[rest]) and (got[gap] == -7).all()
    av, cv, ov, y = dev(a, act), dev(counts), dev(offsets), torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_expert_gemm_packed(p, w.format, K, N, av, None, w.dev, cv, ov, y)
    for _ in range(3):
        y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    # segments that reach beyond the rows are cut, sources clamped
    src = torch.full((n,), 1 << 30, dtype=torch.int32, device="cuda")
    src[0] = -5
    far = torch.full((E,), 1 << 30, dtype=torch.int32, device="cuda")
    y = torch.full((n + 8, N), -7.0, dtype=torch.bfloat16, device="cuda")
    B.moe_expert_gemm_packed(p, w.format, K, N, av, src, w.dev, far, ov, y)
    torch.cuda.synchronize()
    assert (y[n:] == -7).all() and torch.isfinite(y[:n]).all()


def test_wide_and_deep():
    check_gemm([2, 1, 4, 1], 1, 4104, 1048, B.MOE_F16, O.INT, 128, False)
    check_gemm([260, 1, 40, 83], 2, 2056, 1048, B.MOE_BF16, O.E2M1, 32, True)
    check_gemm([4] * 1024, 2, 40, 16, B.MOE_BF16, O.E2M1, 64, True)
    check_gemm([40] * 1000, 2, 40, 16, B.MOE_F16, O.INT, 64, True)


@pytest.mark.parametrize("codes,group", [(O.INT, 64), (O.E2M1, 32)])
def test_many_tiles_of_few_rows(codes, group):
    """Blocks of four tiles, the last of an expert past its end, rows of 17 too."""
    counts = [1, 0, 17, 2] * 256
    check_gemm(counts, 2, 72, 168, B.MOE_F16, codes, group, True)
    check_gemm(counts, 2, 264, 112, B.MOE_BF16, codes, group, False, swiglu=True)


@pytest.mark.parametrize("counts", [[5, 8, 3], [300, 100, 4]])
@pytest.mark.parametrize("codes", [O.INT, O.E2M1])
def test_rows_are_their_own(counts, codes):
    """A row that is not finite changes no other, nor do rows left out of the
    segments; results repeat bit for bit, on another stream too."""
    rng = np.random.default_rng(1)
    counts = np.asarray(counts, np.int32)
    n, K, N, act = int(counts.sum()), 264, 72, B.MOE_BF16
    offsets = (np.cumsum(counts) - counts).astype(np.int32)
    p = B.make_problem(n, 3, 1, 8, 1, act)
    a = bits16(rng, (n, K), act)
    w = Weights(rng, 3, N, K, codes, 64, act)

    def run(a, counts, stream=None):
        y = torch.full((n, N), -7.0, dtype=torch.bfloat16, device="cuda")
        args = dev(a, act), None, w.dev, dev(counts), dev(offsets), y
        torch.cuda.synchronize()
        B.moe_expert_gemm_packed(p, w.format, K, N, *args, stream)
        torch.cuda.synchronize()
        return y

    want = run(a, counts)
    bad = a.copy()
    bad[2, K - 1], bad[6, 3] = 0x7fc0, 0x7f80
    got = run(bad, counts, torch.cuda.Stream())
    rest = [r for r in range(n) if r not in (2, 6)]
    assert torch.equal(got[rest], want[rest]) and torch.isnan(got[2]).all() and not torch.isfinite(got[6]).any()
    fewer = counts.copy()
    fewer[0] -= 2
    got = run(a, fewer)
    gap = list(range(int(counts[0]) - 2, int(counts[0])))
    rest = [r for r in range(n) if r not in gap]
    assert torch.equal(got[rest], want[rest]) and (got[gap] == -7).all()


@pytest.mark.parametrize("T", [8, 400])
def test_bad_segments_and_sources_stay_inside(T):
    """Counts and offsets that reach beyond the rows are cut, sources clamped."""
    say(f"[case] packed product with bad tables T={T}")
    rng = np.random.default_rng(2)
    K, N, act, E = 64, 24, B.MOE_F16, 3
    p = B.make_problem(T, E, 1, 8, 1, act)
    w = Weights(rng, E, N, K, O.INT, 32, act)
    a = dev(bits16(rng, (T, K), act), act)
    src = torch.full((T,), 1 << 30, dtype=torch.int32, device="cuda")
    src[0] = -5
    y = torch.full((T + 8, N), -7.0, dtype=torch.float16, device="cuda")
    counts = torch.tensor([1 << 30, -3, 5], dtype=torch.int32, device="cuda")
    offsets = torch.tensor([-4, 2, T - 1], dtype=torch.int32, device="cuda")
    B.moe_expert_gemm_packed(p, w.format, K, N, a, src, w.dev, counts, offsets, y)
    torch.cuda.synchronize()
    assert (y[T:] == -7).all() and torch.isfinite(y).all()


@pytest.mark.parametrize("counts", [[5, 8, 3], [300, 100, 4]])
def test_graph(counts):
    rng = np.random.default_rng(3)
    counts = np.asarray(counts, np.int32)
    n, K, I, act = int(counts.sum()), 264, 48, B.MOE_F16
    offsets = dev((np.cumsum(counts) - counts).astype(np.int32))
    p = B.make_problem(n, 3, 1, 8, 1, act)
    w = Weights(rng, 3, 2 * I, K, O.INT, 128, act)
    a, c = dev(bits16(rng, (n, K), act), act), dev(counts)
    y = torch.empty(n, I, dtype=torch.float16, device="cuda")
    call = lambda: B.moe_expert_gemm_swiglu_packed(p, w.format, K, I, a, None, w.dev, c, offsets, y)  # noqa: E731
    call()
    torch.cuda.synchronize()
    want = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_weights_past_four_gigabytes():
    """The last expert's weights lie past 2^32 bytes, and rows past 2^31 values."""
    say("[case] packed product, 70 experts of 8192 x 16384")
    E, N, K, act = 70, 8192, 16384, B.MOE_BF16
    rng = np.random.default_rng(5)
    one = Weights(rng, 1, N, K, O.E2M1, 128, act)
    w = torch.zeros(E, one.bytes.size, dtype=torch.uint8, device="cuda")
    w[E - 1] = one.dev[0]
    for rows in (3, 140000):
        p = B.make_problem(rows, E, 1, 8, 1, act)
        a = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
        last = bits16(rng, (3, K), act)
        a[rows - 3:] = dev(last, act)
        counts, offsets = torch.zeros(E, dtype=torch.int32, device="cuda"), torch.zeros(E, dtype=torch.int32, device="cuda")
        counts[E - 1], offsets[E - 1] = rows, 0
        y = torch.empty(rows, N, dtype=torch.bfloat16, device="cuda")
        B.moe_expert_gemm_packed(p, one.format, K, N, a, None, w, counts, offsets, y)
        torch.cuda.synchronize()
        v, mag = one.both(0)
        av = oracle.decode16(last, act).astype(np.float64)
        z, dz = av @ v[-64:].T, (K + K / 32 + 8) * 2 * U * (np.abs(av) @ mag[-64:].T)
        assert_within(f64(y[rows - 3:, -64:]), z, dz + round_bound(np.abs(z) + dz, act), f"{rows} rows")
        assert not y[:rows - 3].any()


def test_counts_of_all_rows_for_all_experts_end_with_the_grid():
    """Tiles of 1024 experts that each claim all of 2^24 rows are more than 32 bits
    hold; the call ends with what segments side by side could have, in bounds."""
    T, E, k, K, N, act = (1 << 20) - 1, 1024, 16, 8, 192, B.MOE_BF16
    n = T * k
    say(f"[case] overlapping segments rows={n} E={E}")
    assert E * (-(-n // 16)) * (N // 64) > 1 << 31 and few_rows(n, E, K, N)
    p = B.make_problem(T, E, k, 8, 1, act)
    w = Weights(np.random.default_rng(5), E, N, K, O.INT, 128, act)
    a = torch.ones(T, K, dtype=torch.bfloat16, device="cuda")
    src = torch.arange(n, dtype=torch.int32, device="cuda")
    y = torch.full((n + 1, N), -7.0, dtype=torch.bfloat16, device="cuda")
    counts = torch.full((E,), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    offsets = torch.zeros(E, dtype=torch.int32, device="cuda")
    B.moe_expert_gemm_packed(p, w.format, K, N, a, src, w.dev, counts, offsets, y)
    torch.cuda.synchronize()
    assert (y[n] == -7).all()
    counts = torch.zeros(E, dtype=torch.int32, device="cuda")
    counts[7] = n  # and counts that the rows allow are all served
    B.moe_expert_gemm_packed(p, w.format, K, N, a, src, w.dev, counts, offsets, y)
    torch.cuda.synchronize()
    v, mag = w.both(7)
    z, dz = v.sum(1), (K + 9) * 2 * U * mag.sum(1)
    want = torch.from_numpy(z).cuda()
    bound = torch.from_numpy(dz + round_bound(np.abs(z) + dz, act)).cuda()
    for part in y[:n].split(1 << 20):
        assert ((part.double() - want).abs() <= bound).all()
    assert (y[n] == -7).all()
