"""The training oracle against something other than itself: torch's AdamW in
fp64, autograd, and differences."""
import numpy as np
import pytest
import torch

from oracle import train


@pytest.mark.parametrize("eps,decay,betas", [(1e-8, 0.1, (0.9, 0.999)), (1e-3, 0.0, (0.5, 0.9)), (1e-6, 0.01, (0.0, 0.0))])
def test_adamw_is_torchs(eps, decay, betas):
    rng = np.random.default_rng(3)
    w = rng.standard_normal(50)
    t = torch.nn.Parameter(torch.from_numpy(w.copy()))
    opt = torch.optim.AdamW([t], lr=1e-2, betas=betas, eps=eps, weight_decay=decay, foreach=False)
    m = v = np.zeros(50)
    for step in range(1, 8):
        g = rng.standard_normal(50)
        t.grad = torch.from_numpy(g * 0.25)
        opt.step()
        w, m, v, _ = train.adamw(w, g, m, v, 1e-2, *betas, eps, decay, step, scale=0.25)
        assert np.allclose(w, t.detach().numpy(), rtol=1e-12, atol=1e-14)


def test_a_zero_gradient_leaves_a_new_weight_but_for_its_decay():
    w, m, v, _ = train.adamw([2.0], [0.0], [0.0], [0.0], 0.1, 0.9, 0.999, 1e-8, 0.5, 1)
    assert w[0] == pytest.approx(2.0 * 0.95) and m[0] == v[0] == 0


@pytest.mark.parametrize("gather", [False, True])
def test_weight_grad_is_autograds(gather):
    rng = np.random.default_rng(4)
    T, E, k, K, N = 9, 4, 2, 5, 6
    idx = rng.integers(0, E - 1, T * k)  # the last expert has no rows
    src = np.argsort(idx, kind="stable")
    counts = np.bincount(idx, minlength=E)
    offsets = np.cumsum(counts) - counts
    a = rng.standard_normal((T if gather else T * k, K))
    dy = rng.standard_normal((T * k, N))
    w = torch.randn(E, N, K, dtype=torch.float64, requires_grad=True)
    rows = torch.from_numpy(a[src // k] if gather else a)
    y = torch.einsum("rnk,rk->rn", w[torch.from_numpy(idx[src])], rows)
    y.backward(torch.from_numpy(dy))
    dw, mag = train.weight_grad(dy, a, src if gather else None, k, counts, offsets, E)
    assert np.allclose(dw, w.grad.numpy(), rtol=1e-13, atol=1e-13)
    assert (np.abs(dw) <= mag + 1e-13).all() and not dw[E - 1].any()
    # and a difference along one weight
    with torch.no_grad():
        w[1, 2, 3] += 1.0
        more = (torch.einsum("rnk,rk->rn", w[torch.from_numpy(idx[src])], rows) - y.detach()) * torch.from_numpy(dy)
    assert float(more.sum()) == pytest.approx(dw[1, 2, 3], rel=1e-12)
