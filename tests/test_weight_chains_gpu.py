"""The weights' operators one after the other as a program runs them, eagerly and as one
replayed graph: the layer on 4-bit weights, and a step of training from routing to
AdamW. Every replay has inputs of its own and has to give, bit for bit, what the eager
calls give on them; eager work runs between the replays."""
import pytest
import torch

from combine_router_topk_amd import binding as B
from combine_router_topk_amd import path as P
from pathcheck import say

pytestmark = pytest.mark.gpu


def equal(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def packed_layer(T, E, k, H, I, act, f, skew=0.0):
    """(buffers, packed weights, inner rows, inputs of a pass)."""
    gen = torch.Generator(device="cuda").manual_seed(T + H)
    rand = lambda *n: torch.randn(n, device="cuda", generator=gen)  # noqa: E731
    p = B.make_problem(T, E, k, H, 1, act)
    dt = B._TORCH_ACT[act]
    w = P.pack_experts(rand(E, 2 * I, H) / H ** 0.5, rand(E, H, I) / I ** 0.5, f)
    b = P.allocate(p, torch.zeros(T, E), torch.zeros(T, H, dtype=dt))
    inputs = [(rand(T, E) - skew * torch.arange(E, device="cuda").float().log1p(), rand(T, H).to(dt)) for _ in range(4)]
    return b, w, torch.empty(T * k, I, dtype=dt, device="cuda"), inputs


@pytest.mark.parametrize("T,E,k,H,I,act,codes,group", [
    (300, 16, 4, 256, 128, B.MOE_F16, B.MOE_PACKED_INT, 64), (2000, 16, 2, 1024, 528, B.MOE_BF16, B.MOE_PACKED_E2M1, 32),
    (1, 8, 2, 128, 64, B.MOE_BF16, B.MOE_PACKED_INT, 128)])
def test_the_layer_on_packed_weights_replays(T, E, k, H, I, act, codes, group):
    say(f"[case] packed layer through the products as a graph, T={T}")
    f = B.make_packed_format(codes, group, act)
    b, w, h, inputs = packed_layer(T, E, k, H, I, act, f, 0.5)
    outs = ("idx", "w", "counts", "src", "pos", "y", "out")

    def load(i):
        b.logits.copy_(inputs[i][0])
        b.x.copy_(inputs[i][1])

    want = []
    for i in range(len(inputs)):
        load(i)
        P.run_layer_packed(b, w, h)
        torch.cuda.synchronize()
        want.append({key: getattr(b, key).clone() for key in outs})
    assert not torch.equal(want[0]["out"], want[1]["out"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.run_layer_packed(b, w, h)
    for i in (2, 0, 3, 1, 1):
        load(i)
        h.fill_(float("nan")), b.y.fill_(float("nan")), b.out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for key in outs:
            assert equal(getattr(b, key), want[i][key]), (i, key)


@pytest.mark.parametrize("T,bits", [(1500, 32), (1500, 8), (200, 32)])
def test_a_training_step_replays(T, bits):
    """Routing, both products and the combine, the combine's gradient, the down weights'
    gradient over two micro-batches (the second added; experts cut into parts at 1500
    tokens), and AdamW with its schedule on the device."""
    say(f"[case] training step as a graph, T={T} bits={bits}")
    E, k, H, I, act = 8, 2, 128, 64, B.MOE_BF16
    f = B.make_packed_format(B.MOE_PACKED_E2M1, 32, act)

    class Run:
        def __init__(self):
            self.b, self.w4, self.h, self.inputs = packed_layer(T, E, k, H, I, act, f, 1.0)
            gen = torch.Generator(device="cuda").manual_seed(5)
            rand = lambda *n: torch.randn(n, device="cuda", generator=gen)  # noqa: E731
            self.douts = [(rand(T, H).bfloat16(), rand(T, H).bfloat16()) for _ in self.inputs]
            self.dout = [torch.empty(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            self.dy, self.dgate = torch.empty_like(self.b.y), torch.empty(T * k, device="cuda")
            self.tr = P.allocate_weight_grad(self.b, H, I)
            assert (self.tr.ws.numel() > 0) == (T >= 1024)
            master = rand(E, H, I) / I ** 0.5
            self.t = dict(w=master.bfloat16(), master=master, g=self.tr.dw, weight_decay=0.1)
            if bits == 8:
                self.t |= {n: torch.zeros(E, H, I, dtype=torch.uint8, device="cuda").view(B.E4M3) for n in ("m", "v")}
                self.t |= {n: torch.zeros(E * H * I // 128, device="cuda") for n in ("m_scale", "v_scale")}
            else:
                self.t |= {n: torch.zeros(E, H, I, device="cuda") for n in ("m", "v")}
            self.plan = B.AdamWTensors([self.t])
            self.control = torch.zeros(3, device="cuda")

        def load(self, i, step):
            self.b.logits.copy_(self.inputs[i][0])
            self.b.x.copy_(self.inputs[i][1])
            for to, d in zip(self.dout, self.douts[i]):
                to.copy_(d)
            self.control.copy_(torch.tensor([1e-2 / step, step, 0.5]))

        def step(self):
            P.run_layer_packed(self.b, self.w4, self.h)
            for n, dout in enumerate(self.dout):
                B.moe_combine_backward(self.b.p, dout, self.b.y, self.b.pos, self.b.w, self.dy, self.dgate)
                P.expert_weight_grad(self.b, self.tr, self.h, None, self.dy, add=n > 0)
            B.moe_adamw_step(B.make_adamw(7.0), self.plan, self.control)

        def state(self):
            return {n: x for n, x in self.t.items() if isinstance(x, torch.Tensor)} | {"out": self.b.out, "dgate": self.dgate}

    eager, replayed = Run(), Run()
    replayed.load(0, 1)
    replayed.control[2] = float("nan")  # a pass before the capture, without its step
    replayed.step()
    torch.cuda.synchronize()
    assert equal(replayed.t["master"], eager.t["master"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed.step()
    for step, i in enumerate((1, 0, 3, 2, 1), 1):
        eager.load(i, step), replayed.load(i, step)
        before = eager.t["master"].clone()
        eager.step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert not torch.equal(before, eager.t["master"])
        for key, x in replayed.state().items():
            assert equal(x, eager.state()[key]), (step, key)
        if step == 1:
            # the gradient of both micro-batches beside fp64 sums over the same rows
            b, expert = eager.b, eager.b.idx.long()[eager.b.src.long()]
            want, size = (torch.zeros(E, H, I, dtype=torch.float64, device="cuda") for _ in range(2))
            gate = b.w.double()[b.src.long()]
            for dout in eager.dout:
                dy = gate[:, None] * dout.double()[b.src.long() // k]
                for e in range(E):
                    r = expert == e
                    want[e] += dy[r].T @ eager.h[r].double()
                    size[e] += dy[r].abs().T @ eager.h[r].double().abs()
            # dy is rounded to bf16 from an fp32 product; each sum has at most T rows in
            # fp32 and parts that are added up, and the second one is added to the first
            bound = size * (2.0 ** -8 * 1.02 + 2 * 2.0 ** -24 * (T + 24)) + 2.0 ** -24 * want.abs()
            assert ((eager.tr.dw.double() - want).abs() <= bound).all()
