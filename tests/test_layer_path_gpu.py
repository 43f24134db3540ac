"""The layer's operators together, as a program uses them: norm, routing,
products and combine against the oracle step by step; the few-token layer
against the same layer by its parts; both replayed as HIP graphs."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from combine_router_topk_amd import binding as B
from combine_router_topk_amd import path as P
from conftest import C_CHECK_LIB
from layercheck import (ACTS, U, assert_within, bits16, check_rows8, codes8, codes_of, dev, f64, host, round_bound,
                        scales)
from oracle import layer as L
from pathcheck import bits_to_tensor, say, tensor_bits
from test_expert_gemm_gpu import lost_in_groups, swiglu_bounds

pytestmark = pytest.mark.gpu
EPS = 1e-6


def test_plain_c_caller_of_the_layer():
    say("[case] plain C caller: norm and gradient, products, few-token layer")
    lib = ctypes.CDLL(C_CHECK_LIB)
    lib.moe_c_abi_check_layer.restype = ctypes.c_int
    assert lib.moe_c_abi_check_layer() == 0


def expert_weights(rng, E, H, I):
    wu, wd = codes8(rng, (E, 2 * I, H)), codes8(rng, (E, H, I))
    su = scales(rng, (E, L.blocks(2 * I), L.blocks(H)), 1 / (110 * H ** 0.5))
    sd = scales(rng, (E, L.blocks(H), L.blocks(I)), 1 / (110 * I ** 0.5))
    return P.ExpertWeights(I, dev(wu), dev(su), dev(wd), dev(sd)), wu, su, wd, sd


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,E,k,H,I,R", [(96, 8, 2, 144, 80, 4), (700, 16, 4, 256, 128, 8), (33, 64, 6, 272, 48, 1)])
def test_norm_route_products_combine(T, E, k, H, I, R, act):
    say(f"[case] layer by its parts T={T} E={E} k={k} H={H} I={I} R={R} act={act}")
    rng = np.random.default_rng(T + H)
    p = B.make_problem(T, E, k, H, R, act)
    x, res, g = bits16(rng, (T, H), act), bits16(rng, (T, H), act), bits16(rng, H, act)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    w, wu, su, wd, sd = expert_weights(rng, E, H, I)
    b = P.allocate(p, torch.from_numpy(logits), torch.empty(T, H, dtype=bits_to_tensor(x, act).dtype))
    l = P.allocate_layer(b, I)
    h = torch.empty_like(b.x)
    P.norm(b, l, dev(x, act), dev(res, act), dev(g, act), EPS, h)
    P.run_layer(b, l, w)
    torch.cuda.synchronize()

    hb, rstd, v = L.rms_norm(x, res, g, EPS, act)
    assert np.array_equal(tensor_bits(h), hb)
    check_rows8(codes_of(l.xq), f64(l.xq_scale), v, 25 * U * np.abs(v), "xq")
    assert_within(f64(b.x), v, round_bound(v, act) + 25 * U * np.abs(v), "x")
    ref = oracle.route_and_layout(T, E, k, R, logits)
    for key in ("idx", "counts", "expert_offsets", "pos", "src"):
        assert np.array_equal(host(getattr(b, key)).ravel(), np.asarray(ref[key]).ravel()), key
    # each product from the 8-bit rows that the step before it wrote
    up = (codes_of(l.xq), f64(l.xq_scale), ref["src"], wu, su, ref["counts"], ref["expert_offsets"])
    hv, dv = swiglu_bounds(up, T, k, H, I)
    check_rows8(codes_of(l.hq), f64(l.hq_scale), hv, dv, "hq")
    down = (codes_of(l.hq), f64(l.hq_scale), None, wd, sd, ref["counts"], ref["expert_offsets"])
    y, mag = L.expert_gemm(*down[:3], k, *down[3:], T * k)
    bound = lost_in_groups(down, k, T * k, H) + (I // 8 + 2 * L.blocks(I) + 2) * 2 * U * mag
    assert_within(f64(b.y), y, bound + round_bound(np.abs(y) + bound, act), "y")
    out = oracle.combine(tensor_bits(b.y), ref["pos"], host(b.w).reshape(T, k), k, act)
    terms = oracle.combine(tensor_bits(b.y) & 0x7fff, ref["pos"], host(b.w).reshape(T, k), k, act)
    assert_within(f64(b.out), out, k * U * terms + round_bound(out, act) + k * U * terms, "out")


def test_expert_down_keeps_y_in_the_activation_format():
    T, E, k, H, I = 20, 4, 2, 128, 64
    rng = np.random.default_rng(2)
    outs = []
    for flags in (0, B.MOE_FLAG_OUT_F32):
        p = B.make_problem(T, E, k, H, 1, B.MOE_BF16, flags)
        rng = np.random.default_rng(2)
        b = P.allocate(p, torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)),
                       bits_to_tensor(bits16(rng, (T, H), B.MOE_BF16), B.MOE_BF16))
        l = P.allocate_layer(b, I)
        w = expert_weights(rng, E, H, I)[0]
        P.norm(b, l, b.x.clone(), None, torch.ones(H, dtype=torch.bfloat16, device="cuda"), EPS)
        P.run_layer(b, l, w)
        torch.cuda.synchronize()
        outs.append((b.y.clone(), b.out.clone()))
    assert torch.equal(outs[0][0].view(torch.int16), outs[1][0].view(torch.int16))
    assert outs[1][1].dtype == torch.float32
    assert torch.equal(outs[1][1].to(torch.bfloat16).view(torch.int16), outs[0][1].view(torch.int16))


@pytest.mark.parametrize("flags", [B.MOE_FLAG_EXACT_SUMS, B.MOE_FLAG_EXACT_SUMS | B.MOE_FLAG_OUT_F32])
def test_expert_down_takes_exact_sums_from_the_problem(flags):
    """The path's y is the fp32 product of the same rows, rounded."""
    T, E, k, H, I = 60, 4, 2, 144, 272
    say(f"[case] path with exact sums flags={flags}")
    rng = np.random.default_rng(3)
    p = B.make_problem(T, E, k, H, 1, B.MOE_BF16, flags)
    b = P.allocate(p, torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)),
                   bits_to_tensor(bits16(rng, (T, H), B.MOE_BF16), B.MOE_BF16))
    l, w = P.allocate_layer(b, I), expert_weights(rng, E, H, I)[0]
    P.norm(b, l, b.x.clone(), None, torch.ones(H, dtype=torch.bfloat16, device="cuda"), EPS)
    P.run_layer(b, l, w)
    y = torch.empty(T * k, H, device="cuda")
    B.moe_expert_gemm(B.make_problem(T, E, k, H, 1, B.MOE_BF16, B.MOE_FLAG_OUT_F32), I, H, l.hq, l.hq_scale, None,
                      w.w_down, w.s_down, b.counts, b.expert_offsets, y)
    torch.cuda.synchronize()
    assert torch.equal(b.y.view(torch.int16).flatten(), y.bfloat16().view(torch.int16).flatten())
    assert b.out.dtype == (torch.float32 if flags & B.MOE_FLAG_OUT_F32 else torch.bfloat16)


@pytest.mark.parametrize("act", ACTS)
def test_few_token_layer_against_its_parts(act):
    """The same weights through the 8-bit path and through the few-token
    layer. The 8-bit path rounds the rows and h to e4m3, half a step of 2^-4
    each: two roundings' root mean square, 2^-4 / sqrt(3) a term, stay under a
    tenth of the output's norm."""
    T, E, k, H, I = 32, 16, 4, 512, 256
    rng = np.random.default_rng(8)
    p = B.make_problem(T, E, k, H, 1, act)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    b = P.allocate(p, torch.from_numpy(logits), bits_to_tensor(bits16(rng, (T, H), act), act))
    l = P.allocate_layer(b, I)
    w = expert_weights(rng, E, H, I)[0]
    P.norm(b, l, b.x.clone(), None, torch.ones(H, dtype=b.x.dtype, device="cuda"), EPS)
    P.run_layer(b, l, w)
    parts, idx, gw = f64(b.out), b.idx.clone(), b.w.clone()
    b.out.zero_()
    P.layer_few_tokens(b, w, P.layer_workspace(b, I))
    torch.cuda.synchronize()
    assert torch.equal(b.idx, idx) and torch.equal(b.w, gw)
    whole = f64(b.out)
    assert np.linalg.norm(parts - whole) <= 0.1 * np.linalg.norm(whole)


def test_graph_replays():
    """Norm, routing, products, combine, the few-token layer and the norm's
    gradient captured once; replayed on new inputs between eager work, each
    replay equal to the eager result."""
    T, E, k, H, I, act = 48, 16, 2, 256, 128, B.MOE_BF16
    rng = np.random.default_rng(10)
    p = B.make_problem(T, E, k, H, 4, act)
    dt = torch.bfloat16
    b = P.allocate(p, torch.zeros(T, E), torch.zeros(T, H, dtype=dt))
    l = P.allocate_layer(b, I)
    w = expert_weights(rng, E, H, I)[0]
    x, res, h = (torch.zeros(T, H, dtype=dt, device="cuda") for _ in range(3))
    g = torch.ones(H, dtype=dt, device="cuda")
    out_few, dx, dg = torch.empty_like(b.out), torch.empty_like(x), torch.empty(H, device="cuda")
    idx2, w2 = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    ws = P.layer_workspace(b, I)
    ws2 = torch.empty(B.moe_rms_norm_workspace_bytes(p), dtype=torch.uint8, device="cuda")

    def step():
        P.norm(b, l, x, res, g, EPS, h)
        P.run_layer(b, l, w)
        B.moe_layer_few_tokens(p, I, b.logits, b.x, w.w_up, w.s_up, w.w_down, w.s_down, idx2, w2, out_few, ws)
        B.moe_rms_norm_backward(p, b.out, res, h, g, l.rstd, dx, dg, ws2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    kept = (b.x, h, l.xq, l.xq_scale, l.hq, l.hq_scale, b.y, b.out, out_few, dx, dg, idx2, w2)
    bits = lambda t: t.contiguous().view(torch.uint8).clone()  # noqa: E731
    for i in range(4):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(i)
        x.copy_(torch.randn(T, H, device="cuda", generator=gen))
        res.copy_(torch.randn(T, H, device="cuda", generator=gen))
        b.logits.copy_(torch.randn(T, E, device="cuda", generator=gen))
        step()
        torch.cuda.synchronize()
        want = [bits(t) for t in kept]
        for t in kept:
            t.view(torch.uint8).zero_()
        graph.replay()
        torch.cuda.synchronize()
        for n, (a, t) in enumerate(zip(want, kept)):
            assert torch.equal(a, bits(t)), (i, n)


def test_two_devices_are_refused():
    """Tensors of one call live on one device (a host without a second GPU
    has none to mix: a tensor off the GPU is refused as such)."""
    p = B.make_problem(2, 1, 1, 64, 1, B.MOE_BF16)
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.moe_rms_norm(p, x, None, g, EPS, None, x.clone(), None, None, None)
    with pytest.raises(ValueError, match="contiguous"):
        B.moe_rms_norm(p, x.t().contiguous().t(), None, g.cuda(), EPS, None, x.clone(), None, None, None)
    with pytest.raises(ValueError, match="elements"):
        B.moe_rms_norm(p, x[:1], None, g.cuda(), EPS, None, x.clone(), None, None, None)
    with pytest.raises(ValueError, match="dtype"):
        B.moe_rms_norm(p, x.half(), None, g.cuda(), EPS, None, x.clone(), None, None, None)
