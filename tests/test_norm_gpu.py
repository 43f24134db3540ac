"""The root-mean-square norm and its gradient on the GPU against the oracle.

Bounds (u = 2^-24): mean(h^2) takes at most 8 fused multiply-adds and 2
additions a lane, 8 in the wave, 16 over the waves, the division and eps: under 40 u; its
square root halves that, and the root, the reciprocal and the products with h
and gamma add one each: v is within 25 u. Of the gradient's sums, mean(u n)
has the same chain and three more roundings a term: 48 u of mean |u n|.
"""
import numpy as np
import pytest
import torch

import oracle
from combine_router_topk_amd import binding as B
from layercheck import (ACTS, U, assert_within, bits16, check_rows8, codes_of, dev, f64, host, round_bound,
                        tensor_bits)
from oracle import layer as L
from pathcheck import say

pytestmark = pytest.mark.gpu
EPS = 1e-5


def problem(T, H, act):
    return B.make_problem(T, 1, 1, H, 1, act)


def run_norm(x, r, g, act, y=True, q=True, eps=EPS, stream=None):
    T, H = x.shape
    t = dev(x, act)
    new = lambda dt, *s: torch.full(s, float("nan"), device="cuda").to(dt)  # noqa: E731
    h = new(t.dtype, T, H) if r is not None else None
    out = dict(h=h, y=new(t.dtype, T, H) if y else None, q=new(B.E4M3, T, H) if q else None,
               s=new(torch.float32, T, L.blocks(H)) if q else None, rstd=new(torch.float32, T))
    B.moe_rms_norm(problem(T, H, act), t, dev(r, act), dev(g, act), eps, h, out["y"], out["q"], out["s"],
                   out["rstd"], stream)
    torch.cuda.synchronize()
    return out


def check_norm(x, r, g, act, eps=EPS, **kw):
    o = run_norm(x, r, g, act, eps=eps, **kw)
    hb, rstd, v = L.rms_norm(x, r, g, eps, act)
    if r is not None:
        assert np.array_equal(tensor_bits(o["h"]), hb)
    assert_within(f64(o["rstd"]), rstd, 23 * U * rstd, "rstd")
    dv = 25 * U * np.abs(v)
    if o["y"] is not None:
        assert_within(f64(o["y"]), v, round_bound(v, act) + dv, "y")
    if o["q"] is not None:
        check_rows8(codes_of(o["q"]), f64(o["s"]), v, dv, "q")
    return o


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,H", [(1, 8), (3, 120), (2, 128), (5, 136), (1, 1024), (70, 1032), (4, 2048), (9, 2056),
                                 (1, 4096), (3, 4104), (6, 8192), (3, 8200), (2, 16384), (2, 16376)])
def test_norm(T, H, act):
    say(f"[case] norm T={T} H={H} act={act}")
    rng = np.random.default_rng(H + T)
    x, r, g = bits16(rng, (T, H), act), bits16(rng, (T, H), act, 2.0), bits16(rng, H, act)
    check_norm(x, r, g, act)
    check_norm(x, None, g, act)
    check_norm(x, r, g, act, q=False)
    check_norm(x, None, g, act, y=False, eps=0.0)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,H", [(13000, 72), (7000, 136), (4099, 2872), (1600, 8200)])
def test_norm_many_rows(T, H, act):
    """More rows than blocks: a block takes several, the next one read ahead;
    in place over x and over the residual too."""
    say(f"[case] norm T={T} H={H} act={act}")
    rng = np.random.default_rng(T)
    x, r, g = bits16(rng, (T, H), act), bits16(rng, (T, H), act, 2.0), bits16(rng, H, act)
    o = check_norm(x, r, g, act)
    p = problem(T, H, act)
    for h_is, y_is in (("x", "r"), ("r", "x")):
        t = {"x": dev(x, act), "r": dev(r, act)}
        q, s = torch.empty(T, H, device="cuda").to(B.E4M3), torch.empty(T, L.blocks(H), device="cuda")
        B.moe_rms_norm(p, t["x"], t["r"], dev(g, act), EPS, t[h_is], t[y_is], q, s, None)
        torch.cuda.synchronize()
        assert torch.equal(t[h_is].view(torch.int16), o["h"].view(torch.int16)), (h_is, y_is)
        assert torch.equal(t[y_is].view(torch.int16), o["y"].view(torch.int16)), (h_is, y_is)
        assert torch.equal(q.view(torch.uint8), o["q"].view(torch.uint8)) and torch.equal(s, o["s"]), (h_is, y_is)


@pytest.mark.parametrize("act", ACTS)
def test_norm_special_rows(act):
    say(f"[case] norm of zeros, of the smallest and largest values, infinities and NaN act={act}")
    rng = np.random.default_rng(1)
    T, H = 6, 392
    xv = rng.standard_normal((T, H)).astype(np.float32)
    xv[0] = 0
    xv[1] *= 6e4 if act == B.MOE_F16 else 1e18
    xv[1] = np.clip(xv[1], -6e4, 6e4) if act == B.MOE_F16 else xv[1]
    xv[2] *= 2.0 ** -20 if act == B.MOE_F16 else 1e-20
    xv[3, 130] = np.inf
    xv[4, 7] = np.nan
    x, g = oracle.encode16(xv, act), bits16(rng, H, act)
    ok = [0, 1, 2, 5]
    o = run_norm(x, None, g, act)
    _, rstd, v = L.rms_norm(x[ok], None, g, EPS, act)
    dv = 25 * U * np.abs(v)
    assert_within(f64(o["y"])[ok], v, round_bound(v, act) + dv, "y")
    check_rows8(codes_of(o["q"])[ok], f64(o["s"])[ok], v, dv, "q")
    s, q = f64(o["s"]), L.decode8(codes_of(o["q"]))
    assert (q[0] == 0).all() and (s[0] == np.float32(2.0 ** -100) / np.float32(448)).all()
    # an infinity makes rstd 0: inf * 0 = NaN in its own block, zeros beside it
    assert np.isnan(s[3, 1]) and (s[3, [0, 2, 3]] == s[0, 0]).all() and f64(o["rstd"])[3] == 0
    assert np.isnan(f64(o["y"])[3, 130]) and (np.delete(f64(o["y"])[3], 130) == 0).all()
    # a NaN makes the whole row NaN
    assert np.isnan(s[4]).all() and np.isnan(f64(o["y"])[4]).all()


@pytest.mark.parametrize("act", ACTS)
def test_norm_in_place(act):
    rng = np.random.default_rng(2)
    T, H = 33, 520
    x, r, g = bits16(rng, (T, H), act), bits16(rng, (T, H), act), bits16(rng, H, act)
    o = run_norm(x, r, g, act)
    p = problem(T, H, act)
    for h_is, y_is in (("x", "r"), ("r", "x"), ("x", None), ("r", None)):
        t = {"x": dev(x, act), "r": dev(r, act), None: torch.empty_like(o["y"])}
        B.moe_rms_norm(p, t["x"], t["r"], dev(g, act), EPS, t[h_is], t[y_is], None, None, None)
        torch.cuda.synchronize()
        assert torch.equal(t[h_is].view(torch.int16), o["h"].view(torch.int16)), (h_is, y_is)
        assert torch.equal(t[y_is].view(torch.int16), o["y"].view(torch.int16)), (h_is, y_is)


def test_norm_writes_its_rows_only_and_takes_a_stream():
    act, T, H = B.MOE_BF16, 5, 136
    rng = np.random.default_rng(4)
    x, g = bits16(rng, (T, H), act), bits16(rng, H, act)
    want = run_norm(x, None, g, act)
    y = torch.full((T + 2, H), 7.0, dtype=torch.bfloat16, device="cuda")
    q = torch.full((T + 2, H), 7.0, device="cuda").to(B.E4M3)
    s, rstd = torch.full((T + 2, 2), 7.0, device="cuda"), torch.full((T + 2,), 7.0, device="cuda")
    xd, gd, side = dev(x, act), dev(g, act), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.moe_rms_norm(problem(T, H, act), xd, None, gd, EPS, None, y, q, s, rstd, side)
    torch.cuda.current_stream().wait_stream(side)
    for got, name in ((y, "y"), (q, "q"), (s, "s"), (rstd, "rstd")):
        assert torch.equal(got[:T].contiguous().view(torch.uint8), want[name].contiguous().view(torch.uint8)), name
        assert (got[T:].float() == 7.0).all(), name
    # no rows: nothing is written
    B.moe_rms_norm(problem(0, H, act), xd, None, gd, EPS, None, y, None, None, None)
    torch.cuda.synchronize()
    assert torch.equal(y[:T].view(torch.int16), want["y"].view(torch.int16))


def run_backward(dy, dh, h, g, rstd, act, **kw):
    T, H = h.shape
    p = problem(T, H, act)
    dx = kw.get("dx") if kw.get("dx") is not None else torch.empty(T, H, dtype=dev(h, act).dtype, device="cuda")
    dg = torch.full((H,), float("nan"), device="cuda")
    ws = torch.full((max(1, B.moe_rms_norm_workspace_bytes(p)),), 255, dtype=torch.uint8, device="cuda")
    d = lambda a: a if isinstance(a, torch.Tensor) else dev(a, act)  # noqa: E731
    B.moe_rms_norm_backward(p, d(dy), d(dh), d(h), d(g), torch.from_numpy(rstd).cuda(), dx, dg, ws)
    torch.cuda.synchronize()
    return dx, dg


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,H", [(1, 8), (3, 128), (70, 1032), (5, 2056), (1, 4096), (2, 16384), (1500, 72),
                                 (2300, 264)])
def test_norm_backward(T, H, act):
    say(f"[case] norm backward T={T} H={H} act={act}")
    rng = np.random.default_rng(T + H)
    h, g, dy, dh = (bits16(rng, s, act) for s in ((T, H), H, (T, H), (T, H)))
    rstd = L.rms_norm(h, None, g, EPS, act)[1].astype(np.float32)
    hv, gv, dyv = (oracle.decode16(a, act).astype(np.float64) for a in (h, g, dy))
    n, u = hv * rstd[:, None], dyv * gv
    r = rstd[:, None].astype(np.float64)
    for d in (dh, None):
        dx, dg = run_backward(dy, d, h, g, rstd, act)
        want, wdg = L.rms_norm_backward(dy, d, h, g, rstd, act)
        mean, mag = (u * n).mean(axis=1, keepdims=True), np.abs(u * n).mean(axis=1, keepdims=True)
        bound = r * (6 * U * (np.abs(u) + np.abs(n * mean)) + 48 * U * np.abs(n) * mag) + 2 * U * np.abs(want)
        assert_within(f64(dx), want, bound + round_bound(np.abs(want) + bound, act), "dx")
        chain = -(-T // 1024) + 64 + 16 + 4
        assert_within(f64(dg), wdg, chain * U * np.abs(dyv * n).sum(axis=0) + 1e-30, "dgamma")
        again = run_backward(dy, d, h, g, rstd, act)
        assert torch.equal(dx.view(torch.int16), again[0].view(torch.int16)) and torch.equal(dg, again[1])
    # in place over dy and over dh
    for over in (dy, dh):
        t = dev(over, act)
        dx, dg2 = run_backward(t if over is dy else dy, t if over is dh else dh, h, g, rstd, act, dx=t)
        first = run_backward(dy, dh, h, g, rstd, act)
        assert torch.equal(dx.view(torch.int16), first[0].view(torch.int16)) and torch.equal(dg2, first[1])


def test_norm_rows_past_four_gib():
    """140000 rows of 16384: 2.3e9 elements, rows on both sides of 2^31
    elements and of 4 GiB against the oracle, forward and backward."""
    say("[case] norm of 140000 rows of 16384")
    T, H, act = 140000, 16384, B.MOE_BF16
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    for part in x.split(20000):
        part.normal_(generator=gen)
    g = bits16(np.random.default_rng(6), H, act)
    gd, p = dev(g, act), problem(T, H, act)
    y, q = torch.empty_like(x), torch.empty(T, H, dtype=torch.uint8, device="cuda").view(B.E4M3)
    s, rstd = torch.empty(T, H // 128, device="cuda"), torch.empty(T, device="cuda")
    B.moe_rms_norm(p, x, None, gd, EPS, None, y, q, s, rstd)
    rows = [0, 131071, 131072, 131073, T - 1]
    xb = np.stack([tensor_bits(x[r]) for r in rows])
    _, want, v = L.rms_norm(xb, None, g, EPS, act)
    pick = lambda t: np.stack([f64(t[r]) for r in rows])  # noqa: E731
    dv = 25 * U * np.abs(v)
    assert_within(np.array([float(rstd[r]) for r in rows]), want, 23 * U * want, "rstd")
    assert_within(pick(y), v, round_bound(v, act) + dv, "y")
    check_rows8(np.stack([codes_of(q[r]) for r in rows]), pick(s), v, dv, "q")
    # backward over y itself as dy, in place
    yb = np.stack([tensor_bits(y[r]) for r in rows])
    dg, ws = torch.empty(H, device="cuda"), torch.empty(B.moe_rms_norm_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    B.moe_rms_norm_backward(p, y, None, x, gd, rstd, y, dg, ws)
    r32 = np.array([float(rstd[r]) for r in rows], np.float32)
    want, _ = L.rms_norm_backward(yb, None, xb, g, r32, act)
    hv, gv, dyv = (oracle.decode16(a, act).astype(np.float64) for a in (xb, g, yb))
    r = r32[:, None].astype(np.float64)
    n, u = hv * r, dyv * gv
    mean, mag = (u * n).mean(axis=1, keepdims=True), np.abs(u * n).mean(axis=1, keepdims=True)
    bound = r * (6 * U * (np.abs(u) + np.abs(n * mean)) + 48 * U * np.abs(n) * mag) + 2 * U * np.abs(want)
    assert_within(pick(y), want, bound + round_bound(np.abs(want) + bound, act), "dx")
    assert torch.isfinite(dg).all()


@pytest.mark.parametrize("T,H", [(140000, 16384), (200003, 1032)])
def test_norm_backward_weight_gradient_of_many_rows(T, H):
    """dgamma over hundreds of rows a block against fp64 sums of the same
    products, and dx of rows on both sides of 2^31 elements."""
    say(f"[case] norm backward T={T} H={H}: dgamma")
    act, p = B.MOE_BF16, problem(T, H, B.MOE_BF16)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(7)
    h, dy = (torch.empty(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for t in (h, dy):
        for part in t.split(20000):
            part.normal_(generator=gen)
    # means, so that the rows of a block add up: a lost block is 10 times the bound
    for part in h.split(20000):
        part += 0.5
    for part in dy.split(20000):
        part += 0.25
    g = dev(bits16(np.random.default_rng(7), H, act), act)
    rstd = torch.rand(T, device="cuda", generator=gen) + 0.5
    dx, dg = torch.empty_like(h), torch.empty(H, device="cuda")
    ws = torch.empty(B.moe_rms_norm_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    B.moe_rms_norm_backward(p, dy, None, h, g, rstd, dx, dg, ws)
    want, mag = (torch.zeros(H, dtype=torch.float64, device="cuda") for _ in range(2))
    for lo in range(0, T, 4000):
        t = dy[lo:lo + 4000].double() * h[lo:lo + 4000].double() * rstd[lo:lo + 4000, None].double()
        want += t.sum(0)
        mag += t.abs().sum(0)
    chain = -(-T // 1024) + 64 + 16 + 4  # a block's rows, the segments, the product's roundings
    assert_within(f64(dg), want.cpu().numpy(), chain * U * mag.cpu().numpy(), "dgamma")
    rows = [0, 131071, 131072, T - 1]
    pick = lambda t: np.stack([f64(t[r]) for r in rows])  # noqa: E731
    hv, dyv, r = pick(h), pick(dy), np.array([[float(rstd[i])] for i in rows])
    n, u = hv * r, dyv * f64(g)
    mean, most = (u * n).mean(axis=1, keepdims=True), np.abs(u * n).mean(axis=1, keepdims=True)
    dxv = r * (u - n * mean)
    bound = r * (6 * U * (np.abs(u) + np.abs(n * mean)) + 48 * U * np.abs(n) * most) + 2 * U * np.abs(dxv)
    assert_within(pick(dx), dxv, bound + round_bound(np.abs(dxv) + bound, act), "dx")


def test_norm_backward_without_rows():
    p = problem(0, 64, B.MOE_BF16)
    dg = torch.full((64,), 3.0, device="cuda")
    B.moe_rms_norm_backward(p, None, None, None, None, None, None, dg, None)
    torch.cuda.synchronize()
    assert (dg == 0).all()


def test_norm_forward_and_backward_against_differences():
    """The two calls together: a loss over y and h, moved by one input."""
    act, T, H = B.MOE_F16, 4, 64
    rng = np.random.default_rng(9)
    x, g, dy, dh = (bits16(rng, s, act) for s in ((T, H), H, (T, H), (T, H)))
    o = run_norm(x, None, g, act, q=False)
    dx, dg = run_backward(dy, dh, x, g, host(o["rstd"]), act)
    hv, gv, dyv, dhv = (oracle.decode16(a, act).astype(np.float64) for a in (x, g, dy, dh))

    def loss(hh, gg):
        v = hh / np.sqrt((hh * hh).mean(axis=1, keepdims=True) + EPS) * gg
        return (v * dyv).sum() + (hh * dhv).sum()

    d = 1e-5
    for i in [(0, 0), (1, 17), (3, 63)]:
        e = np.zeros((T, H))
        e[i] = d
        want = (loss(hv + e, gv) - loss(hv - e, gv)) / (2 * d)
        assert abs(f64(dx)[i] - want) <= 2.0 ** -11 * abs(want) + 1e-5
        e = np.zeros(H)
        e[i[1]] = d
        want = (loss(hv, gv + e) - loss(hv, gv - e)) / (2 * d)
        assert abs(f64(dg)[i[1]] - want) <= 1e-5 * (1 + abs(want))
