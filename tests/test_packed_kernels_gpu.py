"""The products with 4-bit weights by the kernel that takes them: the cases meant for
many rows do reach the kernel of many rows, at one, two and more steps of K, and tables
out of range give what clamping them gives, on both kernels."""
import numpy as np
import pytest
import torch

import oracle
from combine_router_topk_amd import binding as B
from graphkernels import kernels_of
from layercheck import ACTS, U, assert_within, bits16, dev, f64, round_bound
from oracle import packed as O
from packedcheck import FORMATS, Weights
from pathcheck import say
from test_packed_gemm_gpu import LARGE, check_gemm

pytestmark = pytest.mark.gpu
MANY_ROWS, FEW_ROWS = "packed_fat_kernel", "packed_thin_kernel"


def kernel(rows, E, K, N, swiglu=False, act=B.MOE_BF16, codes=O.INT, group=64):
    """The kernel that takes `rows` rows of E experts' [N, K] (swiglu: [2 N, K])."""
    p, f = B.make_problem(rows, E, 1, 8, 1, act), B.make_packed_format(codes, group, act)
    dt = torch.float16 if act == B.MOE_F16 else torch.bfloat16
    a, y = (torch.empty(rows, n, dtype=dt, device="cuda") for n in (K, N))
    w = torch.empty(B.moe_packed_weight_bytes(f, E, 2 * N if swiglu else N, K), dtype=torch.uint8, device="cuda")
    tables = torch.zeros(2, E, dtype=torch.int32, device="cuda")
    f_call = B.moe_expert_gemm_swiglu_packed if swiglu else B.moe_expert_gemm_packed
    names = kernels_of(lambda: f_call(p, f, K, N, a, None, w, tables[0], tables[1], y))
    assert len(names) == 1, names
    return next(k for k in (MANY_ROWS, FEW_ROWS) if k in names[0])


# counts, k, K, N, swiglu: three steps of K (the last one short), four, two (whole and
# short) and one
MANY = [(LARGE, 2, 264, 4104, False), (LARGE, 2, 392, 4112, False), (LARGE, 2, 264, 2064, True), (LARGE, 1, 264, 4104, False),
        (LARGE, 2, 256, 4104, False), (LARGE, 3, 160, 8200, False), (LARGE, 2, 256, 2064, True), (LARGE, 2, 168, 4112, True),
        ([40] * 300, 2, 128, 2056, False), ([40] * 300, 3, 104, 2056, False), ([150] * 40, 2, 128, 2064, True)]


@pytest.mark.parametrize("counts,k,K,N,swiglu", MANY)
def test_many_rows_take_the_kernel_of_many_rows(counts, k, K, N, swiglu):
    for act, codes, group in ((B.MOE_F16, O.INT, 128), (B.MOE_BF16, O.E2M1, 32)):
        assert kernel(sum(counts), len(counts), K, N, swiglu, act, codes, group) == MANY_ROWS


def test_few_rows_take_the_other():
    for rows, E, K, N, swiglu in ((1, 1, 8, 8, False), (64, 64, 4096, 2048, False), (2048, 256, 4096, 2048, True)):
        assert kernel(rows, E, K, N, swiglu) == FEW_ROWS


@pytest.mark.parametrize("codes,group", FORMATS)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("counts,k,K,N,swiglu", MANY[4:8] + MANY[10:])
def test_one_and_two_steps_of_many_rows(counts, k, K, N, swiglu, act, codes, group):
    assert kernel(sum(counts), len(counts), K, N, swiglu, act, codes, group) == MANY_ROWS
    check_gemm(counts, k, K, N, act, codes, group, gather=True, swiglu=swiglu)


@pytest.mark.parametrize("T,k,E,K,N,name", [(9, 1, 3, 64, 24, FEW_ROWS), (400, 2, 3, 264, 72, FEW_ROWS),
                                            (2442, 1, 24, 264, 4104, MANY_ROWS), (1221, 2, 24, 256, 4104, MANY_ROWS)])
@pytest.mark.parametrize("codes", [O.INT, O.E2M1])
def test_tables_out_of_range_give_what_clamping_gives(T, k, E, K, N, name, codes):
    """One expert's count and offset far out on both sides, one negative, one cut at the
    end of the rows; sources below and above the rows."""
    n, act = T * k, B.MOE_F16
    assert kernel(n, E, K, N, act=act, codes=codes, group=32) == name
    say(f"[case] packed product, tables out of range, rows={n} {name}")
    rng = np.random.default_rng(n)
    p = B.make_problem(T, E, k, 8, 1, act)
    w = Weights(rng, E, N, K, codes, 32, act)
    a = bits16(rng, (T, K), act)
    src = torch.full((n,), 1 << 30, dtype=torch.int32, device="cuda")
    src[0], src[1], src[2] = -5, -(1 << 31), n - 1
    src[3] = k * (T // 2)
    token = np.full(n, T - 1)
    token[0] = token[1] = 0
    token[3] = T // 2
    counts, offsets = torch.zeros(2, E, dtype=torch.int32, device="cuda")
    half = n // 2
    # expert 0 the first half, 1 none, 2 the second half and beyond, the last one none
    counts[0], offsets[0] = half, -4
    counts[1], offsets[1] = -3, 2
    counts[2], offsets[2] = 2 ** 31 - 1, half
    counts[E - 1], offsets[E - 1] = (2 ** 31 - 1, half) if E == 3 else (7, 2 ** 31 - 1)
    y = torch.full((n + 8, N), -7.0, dtype=torch.float16, device="cuda")
    B.moe_expert_gemm_packed(p, w.format, K, N, dev(a, act), src, w.dev, counts, offsets, y)
    torch.cuda.synchronize()
    av = oracle.decode16(a, act).astype(np.float64)[token]
    for e, rows in ((0, slice(0, half)), (2, slice(half, n))):
        v, mag = w.both(e)
        z, dz = av[rows] @ v.T, (K + K / 32 + 8) * 2 * U * (np.abs(av[rows]) @ mag.T)
        assert_within(f64(y[:n])[rows], z, dz + round_bound(np.abs(z) + dz, act), f"rows of expert {e}")
    assert (y[n:] == -7).all()
    # a count past the end with an offset below the rows: all rows are the expert's
    counts.zero_(), offsets.zero_()
    counts[0], offsets[0] = 1 << 30, -(1 << 31)
    y.fill_(-7.0)
    B.moe_expert_gemm_packed(p, w.format, K, N, dev(a, act), src, w.dev, counts, offsets, y)
    torch.cuda.synchronize()
    v, mag = w.both(0)
    z, dz = av @ v.T, (K + K / 32 + 8) * 2 * U * (np.abs(av) @ mag.T)
    assert_within(f64(y[:n]), z, dz + round_bound(np.abs(z) + dz, act), "rows of the only expert")
    assert (y[n:] == -7).all()
