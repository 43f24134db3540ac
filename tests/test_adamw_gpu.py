"""The AdamW step on the GPU against the oracle in fp64.

Bounds (u = 2^-24, half a step of fp32): m is off by at most 6 u of its two
terms' magnitudes (b1, 1 - b1, three products, a sum), v by 8 u. The update takes
those through a root (half of v's), the two corrections (an argument rounded
twice and expm1, at most 2 steps of fp32, or 4 u: 6 u each, half of it under the
root), and about ten more roundings: 32 u of the update's terms in all; w adds
two roundings of its own and, in 16 bits, one of the format. 8-bit states are
held to half a step of their codes around m, or the root of v, as layercheck
does it."""
import numpy as np
import pytest
import torch

from combine_router_topk_amd import binding as B
from layercheck import HALF, TINY16, U, assert_within, check_rows8, codes_of, f64
from oracle import layer as L
from oracle import train
from pathcheck import say

pytestmark = pytest.mark.gpu

DTYPE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ACT = {"f16": B.MOE_F16, "bf16": B.MOE_BF16}
GUARD = 64  # elements behind each array that stay as they were


def room(v, dtype):
    """v on the GPU with a guard behind it: (the array, all of it)."""
    t = torch.from_numpy(np.asarray(v, np.float32))
    whole = torch.full((t.numel() + GUARD,), 7.0).to(dtype).cuda()
    whole[:t.numel()] = t.to(dtype).cuda()
    return whole[:t.numel()], whole


class Case:
    def __init__(self, sizes, w, g, master, bits, seed=0, spread=1.0):
        rng = np.random.default_rng(seed)
        self.bits, self.w_type, self.g_type, self.master = bits, w, g, master
        self.wholes, self.tensors = [], []
        for i, n in enumerate(sizes):
            size = np.exp(rng.standard_normal(-(-n // 128)) * spread).repeat(128)[:n] * 1e-3
            t = dict(weight_decay=[0.1, 0.0, 0.02][i % 3])
            wv = rng.standard_normal(n)
            arrays = [("w", wv, DTYPE[w]), ("g", rng.standard_normal(n) * size, DTYPE[g])]
            if master:
                arrays.append(("master", wv, torch.float32))
            if bits == 32:
                arrays += [("m", rng.standard_normal(n) * size, torch.float32),
                           ("v", (rng.random(n) + 0.05) * size ** 2, torch.float32)]
            for key, v, dtype in arrays:
                t[key], whole = room(v, dtype)
                self.wholes.append((key, n, whole))
            if bits == 8:  # zeros, the state before the first step
                for key in ("m", "v"):
                    t[key], whole = room(np.zeros(n), B.E4M3)
                    t[key + "_scale"], scales = room(np.zeros(L.blocks(n)), torch.float32)
                    self.wholes += [(key, n, whole), (key + "_scale", L.blocks(n), scales)]
            self.tensors.append(t)
        self.plan = B.AdamWTensors(self.tensors)

    def new_grads(self, rng, size=1e-3):
        for t in self.tensors:
            t["g"].copy_(torch.from_numpy((rng.standard_normal(t["g"].numel()) * size).astype(np.float32)))

    def values(self):
        """The tensors as the oracle takes them."""
        out = []
        for t in self.tensors:
            m, v = f64(t["m"]), f64(t["v"])
            if self.bits == 8:
                m = train.state8(codes_of(t["m"]), f64(t["m_scale"]))
                v = train.state8(codes_of(t["v"]), f64(t["v_scale"])) ** 2
            out.append((f64(t["master"] if self.master else t["w"]), f64(t["g"]), m, v, t["weight_decay"]))
        return out

    def check(self, before, h, lr, step, scale):
        """One step was made from `before`."""
        b1, b2 = h.beta1, h.beta2
        for t, (w, g, m, v, decay) in zip(self.tensors, before):
            n = w.size
            if not n:
                continue
            want, wm, wv, size = train.adamw(w, g, m, v, lr, b1, b2, np.float64(np.float32(h.eps)),
                                             np.float64(np.float32(decay)), step, scale)
            dm = 6 * U * (b1 * np.abs(m) + (1 - b1) * np.abs(g * scale)) + 2.0 ** -149
            dv = 8 * U * wv + 2.0 ** -148
            if self.bits == 8:
                check_rows8(codes_of(t["m"])[None], f64(t["m_scale"])[None], wm[None], (dm + U * np.abs(m))[None], "m")
                root, s = np.sqrt(wv), L.spread(f64(t["v_scale"]), n)
                # a root above zero takes at least the smallest code
                small = (root > 0) & (root < s * 2.0 ** -9 * 1.01)
                assert (codes_of(t["v"])[small] == 1).all() or not small.any()
                check_rows8(codes_of(t["v"])[None], f64(t["v_scale"])[None], np.where(small, s * 2.0 ** -9, root)[None],
                            (7 * U * root)[None], "v")
            else:
                assert_within(f64(t["m"]), wm, dm, "m")
                assert_within(f64(t["v"]), wv, dv, "v")
            dw = 32 * U * size + 2 * U * (np.abs(w) + np.abs(lr * decay * w))
            if self.master:
                assert_within(f64(t["master"]), want, dw, "master")
                assert torch.equal(t["w"], t["master"].to(t["w"].dtype)), "w is not its master's rounding"
            elif self.w_type == "f32":
                assert_within(f64(t["w"]), want, dw, "w")
            else:
                act = ACT[self.w_type]
                assert_within(f64(t["w"]), want, dw + HALF[act] * np.abs(want) * (1 + HALF[act]) + TINY16[act], "w")
        for key, n, whole in self.wholes:
            assert (whole[n:].float() == 7.0).all(), f"{key}: written behind its end"


TYPES = [("f32", "f32", False), ("f32", "bf16", False), ("f32", "f16", False), ("bf16", "bf16", True),
         ("f16", "f16", True), ("bf16", "f32", True), ("f16", "f32", False), ("bf16", "bf16", False)]
SIZES = [1, 7, 8, 9, 0, 127, 128, 129, 1000, 2047, 2048, 8191, 8192, 8193, 20011]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("w,g,master", TYPES)
def test_three_steps(w, g, master, bits):
    say(f"[case] adamw {w} {g} master={master} bits={bits}")
    c = Case(SIZES, w, g, master, bits)
    rng = np.random.default_rng(5)
    for step in range(1, 4):
        before = c.values()
        h = B.make_adamw(1e-2, 0.9, 0.99, 1e-8, step)
        B.moe_adamw_step(h, c.plan)
        torch.cuda.synchronize()
        c.check(before, h, np.float64(np.float32(1e-2)), step, 1.0)
        c.new_grads(rng)


@pytest.mark.parametrize("count", [56, 57, 200])
@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_a_launch_holds(count, bits):
    say(f"[case] adamw {count} tensors bits={bits}")
    c = Case([(i * 37) % 300 + (9000 if i % 50 == 3 else 0) for i in range(count)], "f32", "f32", False, bits)
    before, h = c.values(), B.make_adamw(1e-3, 0.9, 0.95, 1e-8, 1)
    B.moe_adamw_step(h, c.plan)
    torch.cuda.synchronize()
    c.check(before, h, np.float64(np.float32(1e-3)), 1, 1.0)


@pytest.mark.parametrize("b1,b2,eps,step,lr", [(0.0, 0.0, 1e-8, 1, 1e-2), (0.9, 0.999, 1e-8, 1, 1e-3),
                                              (0.9, 0.999, 1e-3, 2, 1e-3), (0.95, 0.9999, 1e-8, 100000, 1e-4),
                                              (0.99, 0.999, 0.0, 7, 0.0), (0.3, 0.2, 1e-8, 3, -1e-3)])
def test_numbers_of_a_step(b1, b2, eps, step, lr):
    say(f"[case] adamw b1={b1} b2={b2} eps={eps} step={step} lr={lr}")
    c = Case([300, 8200], "f32", "f32", False, 32, seed=3)
    before, h = c.values(), B.make_adamw(lr, b1, b2, eps, step)
    B.moe_adamw_step(h, c.plan)
    torch.cuda.synchronize()
    c.check(before, h, np.float64(np.float32(lr)), step, 1.0)


def test_wide_blocks_in_8_bits():
    """Values spread over e^8 and more within neighbouring blocks, roots below
    the smallest code, and elements whose gradient is zero."""
    say("[case] adamw wide blocks")
    c = Case([5000], "f32", "f32", False, 8, spread=8.0)
    rng = np.random.default_rng(1)
    for step in range(1, 6):
        g = np.exp(rng.standard_normal(5000) * 6) * rng.choice([-1, 0, 1], 5000)
        c.tensors[0]["g"].copy_(torch.from_numpy(g.astype(np.float32)))
        before, h = c.values(), B.make_adamw(1e-3, 0.9, 0.99, 1e-8, step)
        B.moe_adamw_step(h, c.plan)
        torch.cuda.synchronize()
        c.check(before, h, np.float64(np.float32(1e-3)), step, 1.0)


@pytest.mark.parametrize("bits", [32, 8])
def test_control_on_the_device_and_skipped_steps(bits):
    say(f"[case] adamw control bits={bits}")
    c = Case([1000, 9000, 3], "bf16", "bf16", True, bits)
    h = B.make_adamw(5.0, 0.9, 0.99, 1e-8, 77)  # lr and step come from the device
    control = torch.tensor([1e-2, 1.0, 0.5], device="cuda")
    before = c.values()
    B.moe_adamw_step(h, c.plan, control)
    torch.cuda.synchronize()
    c.check(before, h, np.float64(np.float32(1e-2)), 1, 0.5)
    for bad in (float("nan"), float("inf"), -float("inf")):
        control.copy_(torch.tensor([1e-2, 2.0, bad]))
        kept = [w.clone() for _, _, w in c.wholes]
        B.moe_adamw_step(h, c.plan, control)
        torch.cuda.synchronize()
        for (key, _, w), k in zip(c.wholes, kept):
            assert torch.equal(w.view(torch.uint8), k.view(torch.uint8)), key


def test_gradients_that_are_not_finite_stay_in_their_block():
    say("[case] adamw non-finite gradients")
    for bits in (32, 8):
        c = Case([1000], "f32", "f32", False, bits)
        c.tensors[0]["g"][300] = float("nan")
        c.tensors[0]["g"][700] = float("inf")
        B.moe_adamw_step(B.make_adamw(1e-3), c.plan)
        torch.cuda.synchronize()
        t = c.tensors[0]
        assert torch.isnan(t["w"]).nonzero().flatten().tolist() == [300, 700]
        if bits == 8:
            for key in ("m_scale", "v_scale"):
                assert torch.isnan(t[key]).nonzero().flatten().tolist() == [2, 5], key
        else:
            assert (~torch.isfinite(t["m"])).nonzero().flatten().tolist() == [300, 700]


def test_new_gradients_elsewhere_and_another_stream():
    say("[case] adamw set_grads and stream")
    c, d = Case([5000, 70], "f32", "f32", False, 32), Case([5000, 70], "f32", "f32", False, 32)
    h = B.make_adamw(1e-3, step=4)
    grads = [t["g"].clone() for t in d.tensors]
    d.plan.set_grads(grads)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    B.moe_adamw_step(h, d.plan, stream=side)
    side.synchronize()
    B.moe_adamw_step(h, c.plan)
    torch.cuda.synchronize()
    for a, b in zip(c.tensors, d.tensors):
        for key in ("w", "m", "v"):
            assert torch.equal(a[key], b[key]), key
    with pytest.raises(ValueError, match="2 tensors"):
        d.plan.set_grads(grads[:1])
    with pytest.raises(ValueError, match="elements"):
        d.plan.set_grads(grads[::-1])


@pytest.mark.parametrize("bits", [32, 8])
def test_graph_with_a_schedule_on_the_device(bits):
    """Replays with the step number and learning rate on the device make the
    steps that eager calls with host numbers make, bit for bit."""
    say(f"[case] adamw graph bits={bits}")
    make = lambda: Case([4097, 300], "bf16", "f32", True, bits)  # noqa: E731
    c, d = make(), make()
    control = torch.tensor([0.0, 1.0, 0.0], device="cuda")
    h = B.make_adamw(9.0)
    graph = torch.cuda.CUDAGraph()
    control[2] = float("nan")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        B.moe_adamw_step(h, c.plan, control)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        B.moe_adamw_step(h, c.plan, control)
    rng = np.random.default_rng(2)
    for step in range(1, 5):
        seed = int(rng.integers(1 << 30))
        for x in (c, d):
            x.new_grads(np.random.default_rng(seed))
        control.copy_(torch.tensor([1e-2 / step, float(step), 1.0]))
        torch.cuda.synchronize()
        graph.replay()
        B.moe_adamw_step(B.make_adamw(np.float32(1e-2 / step), step=step), d.plan)
        torch.cuda.synchronize()
        for a, b in zip(c.tensors, d.tensors):
            for key in a:
                if isinstance(a[key], torch.Tensor) and key != "g":
                    assert torch.equal(a[key].view(torch.uint8), b[key].view(torch.uint8)), (step, key)


def test_past_four_gigabytes():
    """A tensor of 2^32 + 300 elements: its last block, and one past 2^31, as a
    small tensor with the same values has them."""
    say("[case] adamw 2^32 + 300 elements")
    n = (1 << 32) + 300
    w = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    m, v = torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.zeros(n, dtype=torch.uint8, device="cuda")
    ms, vs = torch.zeros(L.blocks(n), device="cuda"), torch.zeros(L.blocks(n), device="cuda")
    at = [0, (1 << 31) - 128, 1 << 31, n - 300]
    torch.manual_seed(1)
    part_w, part_g = (torch.randn(300, device="cuda").to(torch.bfloat16) for _ in range(2))
    for i in at:
        w[i:i + 300], g[i:i + 300] = part_w, part_g
    plan = B.AdamWTensors([dict(w=w, g=g, m=m.view(B.E4M3), v=v.view(B.E4M3), m_scale=ms, v_scale=vs)])
    B.moe_adamw_step(B.make_adamw(1e-2), plan)
    sm, sv = torch.zeros(300, dtype=torch.uint8, device="cuda"), torch.zeros(300, dtype=torch.uint8, device="cuda")
    sw, ss = part_w.clone(), torch.zeros(2, 3, device="cuda")
    B.moe_adamw_step(B.make_adamw(1e-2), B.AdamWTensors([dict(w=sw, g=part_g, m=sm.view(B.E4M3), v=sv.view(B.E4M3),
                                                              m_scale=ss[0], v_scale=ss[1])]))
    torch.cuda.synchronize()
    for i in at[:1] + at[2:]:  # whole blocks of their own
        assert torch.equal(w[i:i + 300], sw) and torch.equal(m[i:i + 300], sm) and torch.equal(v[i:i + 300], sv), i
        assert torch.equal(ms[i // 128:i // 128 + 3], ss[0]) and torch.equal(vs[i // 128:i // 128 + 3], ss[1]), i
    assert not w[1000:1 << 20].any()


def test_plain_c_caller():
    import ctypes
    from conftest import C_CHECK_LIB
    say("[case] plain C caller: what trains weights")
    check = ctypes.CDLL(C_CHECK_LIB).moe_c_abi_check_weights
    check.restype = ctypes.c_int
    assert check() == 0


@pytest.mark.parametrize("bits", [32, 8])
def test_states_are_those_of_elementary_operations(bits):
    """Bit for bit what the formulas give one fp32 operation at a time."""
    say(f"[case] adamw states bit for bit, bits={bits}")
    n, b1, b2 = 128 * 4000, 0.9, 0.999
    torch.manual_seed(7)
    size = torch.exp(torch.randn(n // 128, device="cuda")).repeat_interleave(128) * 1e-3
    t = dict(w=torch.zeros(n, device="cuda"), g=torch.empty(n, device="cuda"))
    if bits == 8:
        t |= {k: torch.zeros(n, dtype=torch.uint8, device="cuda").view(B.E4M3) for k in ("m", "v")}
        t |= {k: torch.zeros(n // 128, device="cuda") for k in ("m_scale", "v_scale")}
    else:
        t |= {k: torch.zeros(n, device="cuda") for k in ("m", "v")}
    ref = {k: v.clone() for k, v in t.items()}
    plan = B.AdamWTensors([t])
    spread = lambda s: s.repeat_interleave(128)  # noqa: E731
    for step in range(1, 5):
        g = torch.randn(n, device="cuda") * size
        t["g"].copy_(g)
        B.moe_adamw_step(B.make_adamw(1e-3, b1, b2, 1e-8, step), plan)
        m, v = (ref["m"], ref["v"]) if bits == 32 else \
            (ref["m"].float() * spread(ref["m_scale"]), (ref["v"].float() * spread(ref["v_scale"])).square())
        m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
        if bits == 32:
            ref["m"], ref["v"] = m, v
        else:
            for key, x in (("m", m), ("v", v.sqrt())):
                s = x.view(-1, 128).abs().amax(1).clamp_min(2.0 ** -100) * (1 / 448)
                q = (x / spread(s)).to(B.E4M3).view(torch.uint8)
                if key == "v":
                    q = torch.where((x > 0) & (q == 0), 1, q).to(torch.uint8)
                ref[key], ref[key + "_scale"] = q.view(B.E4M3), s
        for key in ref:
            if key not in ("w", "g"):
                assert torch.equal(t[key].view(torch.uint8), ref[key].view(torch.uint8)), (step, key)
