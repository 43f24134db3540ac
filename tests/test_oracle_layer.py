"""Pins for the oracle of the layer around the routing (no GPU): the e4m3
table and rounding against torch's own type, hand-worked 8-bit rows, the
norm's gradient against differences, the products and the layer against
plain loops on tiny inputs."""
import numpy as np
import pytest
import torch

import oracle
import synth
from oracle import layer as L

F16, BF16 = synth.F16, synth.BF16


def test_e4m3_table_is_torchs():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(L.decode8(codes), want.astype(np.float64), equal_nan=True)


def test_e4m3_rounding_is_torchs():
    rng = np.random.default_rng(0)
    t = np.concatenate([rng.uniform(-448, 448, 4000), rng.normal(0, 1, 4000), rng.normal(0, 0.01, 4000),
                        [0.0, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0, 447.9, 2.0 ** -6, 2.0 ** -7]]).astype(np.float32)
    want = torch.from_numpy(t).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(L.round_e4m3(t.astype(np.float64)), want.astype(np.float64))


def test_quantise_handworked():
    v = np.zeros((3, 130))
    v[0, :3] = [448.0, -1.0, 17.0]      # scale 1: 17 is half way between 16 and 18, to even 16
    v[0, 128:] = [-7.0, 3.5]            # scale 1 / 64
    v[1, 5] = np.inf
    n, s = L.quantise(v)
    assert n[0, :3].tolist() == [448.0, -1.0, 16.0] and s[0].tolist() == [1.0, 7.0 / 448]
    assert n[0, 128:].tolist() == [-448.0, 224.0]
    assert np.isnan(s[1, 0]) and s[1, 1] == 2.0 ** -100 / 448
    assert (s[2] == 2.0 ** -100 / 448).all() and (n[2] == 0).all()


@pytest.mark.parametrize("act", [F16, BF16])
def test_norm_gradient_against_differences(act):
    rng = np.random.default_rng(3)
    T, H, eps = 3, 16, 1e-3
    enc = lambda a: oracle.encode16(a.astype(np.float32), act)  # noqa: E731
    h, g, dy, dh = (enc(rng.normal(size=s)) for s in ((T, H), H, (T, H), (T, H)))
    _, rstd, _ = L.rms_norm(h, None, g, eps, act)
    dx, dg = L.rms_norm_backward(dy, dh, h, g, rstd, act)
    hv, gv, dyv, dhv = (oracle.decode16(a, act).astype(np.float64) for a in (h, g, dy, dh))

    def loss(hh, gg):
        v = hh / np.sqrt((hh * hh).mean(axis=1, keepdims=True) + eps) * gg
        return (v * dyv).sum() + (hh * dhv).sum()

    d = 1e-5
    for i in np.ndindex(T, H):
        e = np.zeros((T, H))
        e[i] = d
        assert abs((loss(hv + e, gv) - loss(hv - e, gv)) / (2 * d) - dx[i]) < 1e-6
    for i in range(H):
        e = np.zeros(H)
        e[i] = d
        assert abs((loss(hv, gv + e) - loss(hv, gv - e)) / (2 * d) - dg[i]) < 1e-6


def test_norm_adds_the_residual_rounded():
    x, r = (oracle.encode16(np.array([[v, 1.0]], np.float32), BF16) for v in (256.0, 1.0))
    h, rstd, v = L.rms_norm(x, r, oracle.encode16(np.ones(2, np.float32), BF16), 0.0, BF16)
    assert oracle.decode16(h, BF16).tolist() == [[256.0, 2.0]]  # 257 to even
    assert np.isclose(rstd[0], 1 / np.sqrt((256.0 ** 2 + 4) / 2)) and np.isclose(v[0, 0], 256 * rstd[0])


@pytest.mark.parametrize("gather", [False, True])
def test_products_against_loops(gather):
    rng = np.random.default_rng(5)
    T, E, k, K, N = 6, 3, 2, 144, 136
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    order = np.argsort(idx.ravel(), kind="stable")
    counts = np.bincount(idx.ravel(), minlength=E)
    offsets = np.cumsum(counts) - counts
    rows = T if gather else T * k
    a = rng.integers(0, 0x7f, (rows, K)).astype(np.uint8)
    w = rng.integers(0, 0x7f, (E, N, K)).astype(np.uint8)
    sa, sw = rng.random((rows, 2)), rng.random((E, 2, 2))
    y, mag = L.expert_gemm(a, sa, order if gather else None, k, w, sw, counts, offsets, T * k)
    for r in range(T * k):
        e = idx.ravel()[order[r]]
        rr = order[r] // k if gather else r
        for n in (0, 127, 128, N - 1):
            want = sum(L.E4M3[a[rr, c]] * sa[rr, c // 128] * L.E4M3[w[e, n, c]] * sw[e, n // 128, c // 128]
                       for c in range(K))
            assert np.isclose(y[r, n], want, rtol=1e-12) and np.isclose(mag[r, n], want, rtol=1e-12)


@pytest.mark.parametrize("act", [F16, BF16])
def test_layer_against_a_loop(act):
    rng = np.random.default_rng(7)
    T, E, k, H, I = 2, 3, 2, 8, 4
    x = oracle.encode16(rng.normal(size=(T, H)).astype(np.float32), act)
    idx, w = np.array([[2, 0], [1, 2]]), np.array([[0.75, 0.25], [0.5, 0.5]], np.float32)
    up, down = rng.normal(size=(E, 2 * I, H)), rng.normal(size=(E, H, I))
    h, v, out = L.moe_layer(x, idx, w, up, down, act)
    xv = oracle.decode16(x, act)
    for t in range(T):
        want = np.zeros(H)
        for j in range(k):
            e = idx[t, j]
            inner = np.array([float(np.dot(up[e, i], xv[t])) for i in range(2 * I)])
            row = np.array([inner[i] / (1 + np.exp(-inner[i])) * inner[I + i] for i in range(I)])
            assert np.allclose(v[t, j], row, rtol=1e-12)
            hv = oracle.decode16(oracle.encode16(row.astype(np.float32), act), act)
            want += float(w[t, j]) * (down[e] @ hv)
        assert np.allclose(out[t], want, rtol=1e-12)
