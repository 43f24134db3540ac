"""AdamW's states bit for bit, in every combination of types: what the header's formulas
give one fp32 operation at a time, with a gradient factor from the device too; and the
weights of the combinations that test_adamw_gpu does not step through."""
import numpy as np
import pytest
import torch

from combine_router_topk_amd import binding as B
from pathcheck import say
from test_adamw_gpu import DTYPE, SIZES, TYPES, Case

pytestmark = pytest.mark.gpu

ALL = [("f32", g, False) for g in DTYPE] + [(w, g, m) for w in ("f16", "bf16") for g in ("f32", w) for m in (False, True)]
OTHERS = [t for t in ALL if t not in TYPES]


def test_all_combinations_are_stepped_through():
    assert len(ALL) == 11 and set(TYPES) < set(ALL) and len(OTHERS) == 3


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("w,g,master", OTHERS)
def test_three_steps(w, g, master, bits):
    say(f"[case] adamw {w} {g} master={master} bits={bits}")
    c = Case(SIZES, w, g, master, bits)
    rng = np.random.default_rng(6)
    for step in range(1, 4):
        before, h = c.values(), B.make_adamw(1e-2, 0.9, 0.99, 1e-8, step)
        B.moe_adamw_step(h, c.plan)
        torch.cuda.synchronize()
        c.check(before, h, np.float64(np.float32(1e-2)), step, 1.0)
        c.new_grads(rng)


def spread(s, n):
    return s.repeat_interleave(128)[:n]


def quantise(x, smallest):
    """(codes, scales) of fp32 x by elementary operations."""
    n = x.numel()
    whole = torch.zeros(-(-n // 128) * 128, device=x.device)
    whole[:n] = x
    s = whole.view(-1, 128).abs().amax(1).clamp_min(2.0 ** -100) * (1 / 448)
    q = (x / spread(s, n)).to(B.E4M3).view(torch.uint8)
    if smallest:
        q = torch.where((x > 0) & (q == 0), 1, q).to(torch.uint8)
    return q, s


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("factor", [None, 1.0, 0.37])
@pytest.mark.parametrize("w,g,master", ALL)
def test_states_are_those_of_elementary_operations(w, g, master, factor, bits):
    """Sizes that are whole chunks of the kernel and ones that end inside a lane's eight,
    over four steps, each from the state before; and nothing in the states depends on the
    weights' types."""
    say(f"[case] adamw states {w} {g} master={master} factor={factor} bits={bits}")
    b1, b2, sizes = 0.9, 0.999, [128 * 500, 20011, 5, 128, 2049]
    gen = torch.Generator(device="cuda").manual_seed(11)
    rand = lambda n: torch.randn(n, device="cuda", generator=gen)  # noqa: E731
    tensors, state = [], []
    for n in sizes:
        wv = rand(n)
        t = dict(w=wv.to(DTYPE[w]), g=torch.zeros(n, dtype=DTYPE[g], device="cuda"), weight_decay=0.1)
        if master:
            t["master"] = wv.clone()
        if bits == 8:
            t |= {k: torch.zeros(n, dtype=torch.uint8, device="cuda").view(B.E4M3) for k in ("m", "v")}
            t |= {k: torch.zeros(-(-n // 128), device="cuda") for k in ("m_scale", "v_scale")}
        else:
            t |= {k: torch.zeros(n, device="cuda") for k in ("m", "v")}
        tensors.append(t)
        state.append([torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")])
    plan = B.AdamWTensors(tensors)
    control = None if factor is None else torch.tensor([1e-3, 0.0, factor], device="cuda")
    for step in range(1, 5):
        for t in tensors:
            n = t["g"].numel()
            size = torch.exp(rand(-(-n // 128))).repeat_interleave(128)[:n] * 1e-2
            t["g"].copy_(rand(n) * size)
        if control is not None:
            control[1] = float(step)
        B.moe_adamw_step(B.make_adamw(1e-3, b1, b2, 1e-8, step), plan, control)
        for i, t in enumerate(tensors):
            n, grad = t["g"].numel(), t["g"].float()
            if factor is not None:
                grad = grad * control[2]
            m, v = state[i]
            m, v = b1 * m + (1 - b1) * grad, b2 * v + (1 - b2) * grad * grad
            if bits == 32:
                want = {"m": m, "v": v}
                state[i] = [m, v]
            else:
                (mq, ms), (vq, vs) = quantise(m, False), quantise(v.sqrt(), True)
                want = {"m": mq, "m_scale": ms, "v": vq, "v_scale": vs}
                state[i] = [mq.view(B.E4M3).float() * spread(ms, n), (vq.view(B.E4M3).float() * spread(vs, n)).square()]
            for key, x in want.items():
                assert torch.equal(t[key].view(torch.uint8), x.view(torch.uint8)), (step, i, key)
            if master:
                assert torch.equal(t["w"], t["master"].to(t["w"].dtype)), (step, i)
