"""Measured cases of what trains the experts' weights and serves them in four
bits: the weights' gradient over the routed rows, an AdamW step over many
tensors with states in 32 or 8 bits, the experts' products and the whole
layer for a few tokens with packed 4-bit weights.

`run` computes each operator in its plain form (elementary torch operations
in 32 bits, rounded once at the end) or, with `own` set, through the package's
entry points. `exact` gives the same outputs from the definitions in 64 bits.

8-bit states hold e4m3 numbers and one f32 scale for each 128 of a tensor;
both are returned. Packed weights come in tiles of 16 rows by 128 columns:
1024 bytes of codes, then 16 rows of 128 / group scales in 16 bits.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
TINY = 2.0 ** -100
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
# of every AdamW case
LR, BETA1, BETA2, EPS, DECAY, STEP = 3e-4, 0.9, 0.95, 1e-8, 0.1, 1000


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # a norm's weight by itself: latency
        dict(name="adamw_one_norm", op="adamw", count=1, big=4096, act="bf16", w16=False, master=False, g16=False,
             bits=32, control=False),
        # a block's experts with its norms and router: 16-bit weights, fp32 masters and states
        dict(name="adamw_experts_32", op="adamw", count=6, big=16 * 4096 * 4096, act="bf16", w16=True, master=True,
             g16=True, bits=32, control=False),
        # the same with 8-bit states, schedule and clipping on the device
        dict(name="adamw_experts_8", op="adamw", count=6, big=16 * 4096 * 4096, act="bf16", w16=True, master=True,
             g16=True, bits=8, control=True),
        # many tensors of odd sizes, fp32 gradients
        dict(name="adamw_many_8", op="adamw", count=150, big=1250003, act="f16", w16=False, master=False, g16=False,
             bits=8, control=True),
        # gate and up weights' gradient of the top-2 batch, token rows through the layout
        dict(name="grad_up_top2", op="grad", T=16384, E=64, k=2, K=4096, N=4096, act="bf16", skew=0.0, gather=True,
             f32=False, add=False),
        # down weights' gradient of the skewed top-6 batch, added up over micro-batches in fp32
        dict(name="grad_down_top6_skewed", op="grad", T=16384, E=64, k=6, K=1024, N=2048, act="bf16", skew=1.2,
             gather=False, f32=True, add=True),
        # odd sizes, few rows
        dict(name="grad_ragged", op="grad", T=1021, E=8, k=2, K=1424, N=2872, act="f16", skew=0.0, gather=True,
             f32=True, add=False),
        # gate and up of a decode batch: every expert's weights for a few rows each
        dict(name="gate_up_decode", op="gate_up", T=256, E=256, k=8, K=4096, I=2048, act="f16", skew=0.0,
             codes="int4", group=128),
        # down product of a prompt's chunk
        dict(name="down_prompt", op="down", T=8192, E=64, k=6, K=1024, N=2048, act="bf16", skew=0.0, codes="e2m1",
             group=32),
        # the whole layer for one decoded token
        dict(name="layer_1_token", op="layer", T=1, E=256, k=8, H=4096, I=2048, act="f16", codes="int4", group=128),
        # the whole layer for a few tokens, widths that end inside a tile
        dict(name="layer_5_tokens_ragged", op="layer", T=5, E=64, k=6, H=2064, I=1424, act="bf16", codes="int4",
             group=64),
        # the whole layer for a decode batch of the widest workload
        dict(name="layer_32_tokens_wide", op="layer", T=32, E=256, k=8, H=7168, I=2048, act="bf16", codes="e2m1",
             group=32),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["adamw", "adamw", "grad", "grad", "gate_up", "down", "layer", "layer"])
    act = rng.choice(["f16", "bf16"])
    if op == "adamw":
        w16 = rng.random() < 0.6
        return dict(op=op, count=_log(rng, 1, 200), big=_log(rng, 100, 10 ** 8), act=act, w16=w16,
                    master=w16 and rng.random() < 0.7, g16=rng.random() < 0.5, bits=rng.choice([8, 32]),
                    control=rng.random() < 0.5)
    if op == "layer":
        E = rng.choice([8, 16, 64, 160, 256])
        return dict(op=op, T=rng.randint(1, 64 if E <= 64 else 32), E=E, k=rng.randint(1, 8),
                    H=_log(rng, 512, 4096, 16), I=_log(rng, 128, 2048, 16), act=act,
                    codes=rng.choice(["int4", "e2m1"]), group=rng.choice([32, 64, 128]))
    E = rng.choice([4, 8, 32, 64, 160])
    k = rng.randint(1, min(E, 8))
    K = _log(rng, 256, 4096, 8)
    skew = rng.choice([0.0, 0.0, 1.2]) if E <= 64 else 0.0
    c = dict(op=op, E=E, k=k, K=K, act=act, skew=skew)
    if op == "gate_up":
        c["I"] = _log(rng, 128, 2048, 16)
        width = 2 * c["I"]
    else:
        c["N"] = _log(rng, 256, 4096, 8)
        width = c["N"]
    if op == "grad":
        c["gather"] = rng.random() < 0.5
        c["f32"] = rng.random() < 0.6
        c["add"] = c["f32"] and rng.random() < 0.4
    else:
        c["codes"], c["group"] = rng.choice(["int4", "e2m1"]), rng.choice([32, 64, 128])
    most = 25 * 10 ** 10 // (k * K * width)  # at most 5e11 operations
    c["T"] = _log(rng, 1, max(1, min(16384, most)))
    return c


def _sizes(c):
    """Elements of each tensor of an AdamW case, the largest first, the others
    spread over the logarithm down to one."""
    return [c["big"]] + [max(1, int(c["big"] ** (i * 0.6180339887 % 1))) for i in range(1, c["count"])]


# ---- inputs ----------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _blocks(n):
    return -(-n // BLOCK)


def _quantise(v):
    """8-bit rows of f32 v: (e4m3 numbers, scales)."""
    p = v.view(-1, BLOCK)
    scale = p.abs().amax(1).clamp_min(TINY) / E4M3_MAX
    return (p / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(-1), scale


def _quantise_root(v):
    """The root of v in 8 bits; one that is not zero takes at least the smallest code."""
    r = v.sqrt()
    q, scale = _quantise(r)
    small = torch.tensor(2.0 ** -9, device=v.device).to(torch.float8_e4m3fn)
    return torch.where((r > 0) & (q.view(torch.uint8) == 0), small, q), scale


def _logits(T, E, skew, g):
    """Router logits; with a skew the experts' popularity falls as a power of their (shuffled) rank."""
    logits = torch.randn(T, E, device="cuda", generator=g)
    if skew:
        rank = torch.randperm(E, device="cuda", generator=g).float() + 1
        logits = logits - skew * torch.log(rank)
    return logits


def _packed(E, rows, cols, c, size, g):
    """Packed weights: codes as a quantised normal weight has them, scales
    around `size` spread over a factor of three; zeros past the matrix."""
    tiles, tile = (E, -(-rows // 16), _blocks(cols)), 1024 + 32 * (BLOCK // c["group"])
    w = torch.empty(*tiles, tile, dtype=torch.uint8, device="cuda")
    flat = w.view(-1, tile)
    for part in flat.split(1 << 17):
        n = part.shape[0]
        v = torch.randn(2, n, 1024, dtype=torch.bfloat16, device="cuda", generator=g)
        if c["codes"] == "int4":
            q = (v * 2.5).round().clamp(-8, 7).add(8).to(torch.uint8)
        else:
            mag = torch.bucketize((v * 2.0).abs().float(), torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.], device="cuda"))
            q = mag.to(torch.uint8) + 8 * (v < 0).to(torch.uint8)
        part[:, :1024] = q[0] | q[1] << 4
        s = ((torch.rand(n, tile // 2 - 512, device="cuda", generator=g) + 0.5) * size).to(DTYPES[c["act"]])
        part[:, 1024:] = s.view(torch.uint8)
    last_r, last_c = tiles[1] * 16 - rows, tiles[2] * BLOCK - cols
    zero = 0x88 if c["codes"] == "int4" else 0
    if last_r:
        t = w[:, -1]
        t[..., :1024].view(E, -1, 4, 16, 16)[:, :, :, 16 - last_r:] = zero
        t[..., 1024:].view(E, -1, 16, tile // 16 - 64)[:, :, 16 - last_r:] = 0
    if last_c:
        t, (col, _) = w[:, :, -1], _columns(c["codes"])
        past = col >= BLOCK - last_c  # of a lane's row: [4, 16 bytes, 2 nibbles]
        keep = torch.where(past[..., 0], 0, 15) + torch.where(past[..., 1], 0, 240)
        fill = torch.where(past[..., 0], zero & 15, 0) + torch.where(past[..., 1], zero & 240, 0)
        codes = t[..., :1024].view(E, -1, 4, 16, 16)
        codes.copy_(codes & keep[:, None].to(torch.uint8) | fill[:, None].to(torch.uint8))
        live = -(-(BLOCK - last_c) // c["group"])
        t[..., 1024:].view(E, -1, 16, tile // 16 - 64)[..., 2 * live:] = 0
    return w


def _columns(codes):
    """Column in its tile of each nibble of a row's chunks: [4 chunks, 16
    bytes, low and high], and the chunk's own axis."""
    g = torch.arange(4, device="cuda")[:, None, None]
    j = (torch.arange(16, device="cuda") // 4)[None, :, None]
    b = (torch.arange(16, device="cuda") % 4)[None, :, None]
    h = torch.arange(2, device="cuda")[None, None, :]
    inner = b + 4 * h if codes == "int4" else 2 * b + h
    return 32 * j + 8 * g + inner, g


def prepare(case, seed):
    g, c = _gen(seed), dict(case)
    op, act = c["op"], DTYPES[c["act"]]
    rand = lambda *s: torch.randn(s, device="cuda", generator=g).to(act)  # noqa: E731
    s = {"case": c}
    if op == "adamw":
        # one buffer of each kind holds all tensors, each from a multiple of 128 on, zeros between them
        sizes = _sizes(c)
        at = [0]
        for n in sizes:
            at.append(at[-1] + _blocks(n) * BLOCK)
        total = at[-1]
        live = torch.zeros(total, dtype=torch.bool, device="cuda")
        for a, n in zip(at, sizes):
            live[a:a + n] = True
        size = torch.exp(torch.randn(total // BLOCK, device="cuda", generator=g)).repeat_interleave(BLOCK) * 1e-3 * live
        w = torch.randn(total, device="cuda", generator=g).mul_(0.02).mul_(live)
        s["w"] = w.to(act) if c["w16"] else w
        s["master"] = w if c["master"] else None
        grad = torch.randn(total, device="cuda", generator=g).mul_(size)
        s["g"] = grad.to(act) if c["g16"] else grad
        m = torch.randn(total, device="cuda", generator=g).mul_(size).mul_(0.25)
        v = torch.rand(total, device="cuda", generator=g).add_(0.1).mul_(size).mul_(size)
        if c["bits"] == 8:
            s["m"], s["m_scale"] = _quantise(m)
            s["v"], s["v_scale"] = _quantise_root(v)
        else:
            s["m"], s["v"] = m, v
        s["sizes"], s["at"] = sizes, at
        s["decay"] = [DECAY if n > 10000 else 0.0 for n in sizes]  # matrices alone
        s["decay_of"] = torch.zeros(total, device="cuda")
        for a, n, d in zip(at, sizes, s["decay"]):
            s["decay_of"][a:a + n] = d
        if c["control"]:
            s["control"] = torch.tensor([LR, STEP, 0.5], device="cuda")
        return s
    if op == "layer":
        T, E, H, I = c["T"], c["E"], c["H"], c["I"]
        s["logits"] = _logits(T, E, 0.0, g)
        s["x"] = rand(T, H)
        s["w_up"] = _packed(E, 2 * I, H, c, 0.4 / math.sqrt(H), g)
        s["w_down"] = _packed(E, H, I, c, 0.4 / math.sqrt(I), g)
        return s
    T, E, k, K = c["T"], c["E"], c["k"], c["K"]
    # the routed batch, as the layout gives it: rows by expert, then by token
    idx = torch.sort(_logits(T, E, c["skew"], g), dim=1, descending=True, stable=True)[1][:, :k]
    s["src"] = torch.argsort(idx.reshape(-1), stable=True).to(torch.int32)
    counts = torch.bincount(idx.reshape(-1), minlength=E)
    s["counts"] = counts.to(torch.int32)
    s["offsets"] = (torch.cumsum(counts, 0) - counts).to(torch.int32)
    if op == "grad":
        s["a"] = rand(T if c["gather"] else T * k, K)
        s["dy"] = torch.randn(T * k, c["N"], device="cuda", generator=g).mul_(0.05).to(act)
        if c["add"]:
            s["dw"] = torch.randn(E, c["N"], K, device="cuda", generator=g)
        return s
    s["a"] = rand(T if op == "gate_up" else T * k, K)
    s["w"] = _packed(E, 2 * c["I"] if op == "gate_up" else c["N"], K, c, 0.4 / math.sqrt(K), g)
    return s


# ---- the plain form ----------------------------------------------------------

def _plain_adamw(s):
    c = s["case"]
    lr, step, scale = s["control"] if c["control"] else (LR, STEP, 1.0)
    g = s["g"].float() * scale
    if c["bits"] == 8:
        m = s["m"].float() * s["m_scale"].repeat_interleave(BLOCK)
        v = (s["v"].float() * s["v_scale"].repeat_interleave(BLOCK)).square()
    else:
        m, v = s["m"], s["v"]
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    w = (s["w"] if s["master"] is None else s["master"]).float()
    step = torch.as_tensor(step, dtype=torch.float64, device="cuda")
    c1, c2 = (1 - BETA1 ** step).float(), (1 - BETA2 ** step).float()
    w = w - (lr * s["decay_of"] * w + lr * (m / c1) / ((v / c2).sqrt() + EPS))
    s["w"].copy_(w)
    out = {"w": s["w"]}
    if s["master"] is not None:
        out["master"] = s["master"].copy_(w)
    if c["bits"] == 8:
        for key, (q, scale) in (("m", _quantise(m)), ("v", _quantise_root(v))):
            out[key], out[key + "_scale"] = s[key].copy_(q), s[key + "_scale"].copy_(scale)
    else:
        out["m"], out["v"] = s["m"].copy_(m), s["v"].copy_(v)
    return out


def _places(s):
    """Expert and place in its segment of every send row."""
    rows = torch.arange(s["src"].numel(), device="cuda")
    expert = torch.bucketize(rows, (s["offsets"] + s["counts"]).long(), right=True)
    return expert, rows - s["offsets"].long()[expert]


def _rows(s, gather):
    a = s["a"].float()
    return a[s["src"].long() // s["case"]["k"]] if gather else a


def _padded(v, expert, place, s):
    """Rows of every expert padded to the longest segment."""
    p = torch.zeros(s["case"]["E"], max(1, int(s["counts"].max())), v.shape[1], device="cuda")
    p[expert, place] = v
    return p


def _plain_grad(s):
    c = s["case"]
    expert, place = _places(s)
    a = _padded(_rows(s, c["gather"]), expert, place, s)
    dy = _padded(s["dy"].float(), expert, place, s)
    dw = torch.bmm(dy.transpose(1, 2), a)
    if c["add"]:
        return {"dw": s["dw"].add_(dw)}
    return {"dw": dw if c["f32"] else dw.to(DTYPES[c["act"]])}


def _unpack(w, rows, cols, c):
    """f32 [n, rows, cols] of packed weights [n, row tiles, column tiles, bytes]."""
    n, nt, kt, _ = w.shape
    b = w[..., :1024].view(n, nt, kt, 4, 16, 4, 4)  # chunk, row, dword, byte
    if c["codes"] == "int4":
        v = torch.cat([b & 15, b >> 4], dim=-1).float().sub_(8)
    else:
        q = torch.stack([b & 15, b >> 4], dim=-1).view(n, nt, kt, 4, 16, 4, 8)
        v = torch.tensor(E2M1, device="cuda")[q.int()]
    v = v.permute(0, 1, 4, 2, 5, 3, 6).reshape(n, nt * 16, kt * BLOCK)  # row; column tile, dword, chunk, place
    per = BLOCK // c["group"]
    scale = w[..., 1024:].contiguous().view(DTYPES[c["act"]]).view(n, nt, kt, 16, per).transpose(2, 3)
    v.view(n, nt * 16, kt * per, c["group"]).mul_(scale.reshape(n, nt * 16, kt * per, 1).float())
    return v[:, :rows, :cols]


def _plain_product(s):
    c = s["case"]
    gather = c["op"] == "gate_up"
    rows = 2 * c["I"] if gather else c["N"]
    expert, place = _places(s)
    a = _padded(_rows(s, gather), expert, place, s)
    z = torch.bmm(a, _unpack(s["w"], rows, c["K"], c).transpose(1, 2))[expert, place]
    if gather:
        z = z[:, :c["I"]] * torch.sigmoid(z[:, :c["I"]]) * z[:, c["I"]:]
    return {"y": z.to(DTYPES[c["act"]])}


def _plain_layer(s):
    c = s["case"]
    top, idx = torch.sort(s["logits"], dim=1, descending=True, stable=True)
    top, idx = top[:, :c["k"]].double(), idx[:, :c["k"]]
    e = torch.exp(top - top[:, :1])
    w = (e / e.sum(1, keepdim=True)).float()
    pick = idx.reshape(-1)
    x = s["x"].float().repeat_interleave(c["k"], dim=0)[:, :, None]
    z = torch.bmm(_unpack(s["w_up"][pick], 2 * c["I"], c["H"], c), x)[:, :, 0]
    gate, up = z[:, :c["I"]], z[:, c["I"]:]
    h = (gate * torch.sigmoid(gate) * up).to(s["x"].dtype).float()
    y = torch.bmm(_unpack(s["w_down"][pick], c["H"], c["I"], c), h[:, :, None])[:, :, 0]
    out = (y.view(c["T"], c["k"], -1) * w[:, :, None]).sum(1)
    return {"idx": idx.to(torch.int32), "w": w, "out": out.to(s["x"].dtype)}


# ---- the package's calls -----------------------------------------------------

def _own(s):
    from combine_router_topk_amd import binding as B
    c = s["case"]
    act = DTYPES[c["act"]]
    fmt = B.MOE_F16 if c["act"] == "f16" else B.MOE_BF16
    new = lambda *shape, dtype=act: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    if c["op"] == "adamw":
        if "plan" not in s:  # the list of tensors, as an optimizer keeps it
            cut = lambda key, i: s[key][s["at"][i]:s["at"][i] + s["sizes"][i]]  # noqa: E731
            blocks = lambda key, i: s[key][s["at"][i] // BLOCK:s["at"][i + 1] // BLOCK]  # noqa: E731
            s["plan"] = B.AdamWTensors(
                [dict(w=cut("w", i), master=cut("master", i) if c["master"] else None, g=cut("g", i), m=cut("m", i),
                      v=cut("v", i), weight_decay=s["decay"][i],
                      **(dict(m_scale=blocks("m_scale", i), v_scale=blocks("v_scale", i)) if c["bits"] == 8 else {}))
                 for i in range(c["count"])])
        B.moe_adamw_step(B.make_adamw(LR, BETA1, BETA2, EPS, STEP), s["plan"], s.get("control"))
        return {key: s[key] for key in ("w", "master", "m", "v", "m_scale", "v_scale") if s.get(key) is not None}
    T, E, k = c["T"], c["E"], c["k"]
    if c["op"] == "grad":
        p = B.make_problem(T, E, k, c["K"], 1, fmt, B.MOE_FLAG_OUT_F32 if c["f32"] else 0)
        dw = s["dw"] if c["add"] else new(E, c["N"], c["K"], dtype=torch.float32 if c["f32"] else act)
        ws = new(B.moe_expert_weight_grad_workspace_bytes(p, c["K"], c["N"]), dtype=torch.uint8)
        B.moe_expert_weight_grad(p, c["K"], c["N"], s["a"], s["src"] if c["gather"] else None, s["dy"], s["counts"],
                                 s["offsets"], c["add"], dw, ws)
        return {"dw": dw}
    f = B.make_packed_format(B.MOE_PACKED_INT if c["codes"] == "int4" else B.MOE_PACKED_E2M1, c["group"], fmt)
    if c["op"] == "layer":
        p = B.make_problem(T, E, k, c["H"], 1, fmt)
        idx, w, out = new(T, k, dtype=torch.int32), new(T, k, dtype=torch.float32), new(T, c["H"])
        ws = new(B.moe_layer_packed_workspace_bytes(p, c["I"]), dtype=torch.uint8)
        B.moe_layer_few_tokens_packed(p, f, c["I"], s["logits"], s["x"], s["w_up"], s["w_down"], idx, w, out, ws)
        return {"idx": idx, "w": w, "out": out}
    p = B.make_problem(T, E, k, c["K"], 1, fmt)
    if c["op"] == "gate_up":
        y = new(T * k, c["I"])
        B.moe_expert_gemm_swiglu_packed(p, f, c["K"], c["I"], s["a"], s["src"], s["w"], s["counts"], s["offsets"], y)
    else:
        y = new(T * k, c["N"])
        B.moe_expert_gemm_packed(p, f, c["K"], c["N"], s["a"], None, s["w"], s["counts"], s["offsets"], y)
    return {"y": y}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "adamw":
        return _plain_adamw(state)
    if op == "grad":
        return _plain_grad(state)
    return _plain_layer(state) if op == "layer" else _plain_product(state)


# ---- what a pass cannot do without -------------------------------------------

def work(case):
    c = case
    if c["op"] == "adamw":
        n = sum(_sizes(c))
        w = (2 + 8 if c["master"] else 4) if c["w16"] else 8
        states = 4 * (1 + 4 / BLOCK) if c["bits"] == 8 else 16
        return {"bytes": int(n * (w + (2 if c["g16"] else 4) + states)), "flops": 16 * n}
    T, E, k = c["T"], c["E"], c["k"]
    rows = T * k
    active = min(E, rows, max(k, round(E * (1 - (1 - k / E) ** T))))
    if c["op"] == "grad":
        K, N = c["K"], c["N"]
        out = E * N * K * (8 if c["add"] else 4 if c["f32"] else 2)
        return {"bytes": out + 2 * (T if c["gather"] else rows) * K + 2 * rows * N + 8 * E + 4 * rows * c["gather"],
                "flops": 2 * rows * K * N}
    per = 0.5 + 2 / c["group"]
    if c["op"] == "layer":
        weights = 3 * c["H"] * c["I"]
        return {"bytes": int(active * weights * per) + 4 * T * E + 4 * T * c["H"] + 8 * rows,
                "flops": 2 * rows * weights}
    K, N, out = (c["K"], 2 * c["I"], c["I"]) if c["op"] == "gate_up" else (c["K"], c["N"], c["N"])
    a_rows = T if c["op"] == "gate_up" else rows
    return {"bytes": int(active * N * K * per) + 2 * a_rows * K + 2 * rows * out + 8 * E + 4 * rows,
            "flops": 2 * rows * K * N}


# ---- the definitions in 64 bits ------------------------------------------------

def _exact_codes(v, smallest):
    """e4m3 numbers and scales of f64 v, 128 at a time."""
    p = v.reshape(-1, BLOCK)
    scale = torch.clamp(p.abs().max(dim=1, keepdim=True).values, min=TINY) / 448
    t = p / scale
    # spacing of e4m3 around t: 2^-3 of its power of two, 2^-9 below 2^-6
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
    q = torch.clamp(torch.round(t / step) * step, -448, 448)
    if smallest:
        q = torch.where((p > 0) & (q == 0), torch.full_like(q, 2.0 ** -9), q)
    return q.reshape(-1), scale.reshape(-1)


def _exact_adamw(s):
    c = s["case"]
    lr, n, scale = s["control"].double().tolist() if c["control"] else (LR, STEP, 1.0)
    names = ["w"] + (["master"] if s["master"] is not None else []) + ["m", "v"]
    names += ["m_scale", "v_scale"] if c["bits"] == 8 else []
    out = {key: torch.zeros(s[key].shape, dtype=torch.float64, device="cuda") for key in names}
    if c["bits"] == 8:
        out["m_scale"] += TINY / 448
        out["v_scale"] += TINY / 448
    for lo, hi, size, decay in zip(s["at"], s["at"][1:], s["sizes"], s["decay"]):
        i, b = slice(lo, hi), slice(lo // BLOCK, hi // BLOCK)
        spread = lambda key: s[key][b].double()[:, None].expand(-1, BLOCK).reshape(-1)  # noqa: E731
        g = scale * s["g"][i].double()
        m, v = s["m"][i].double(), s["v"][i].double()
        if c["bits"] == 8:
            m, v = m * spread("m_scale"), torch.pow(v * spread("v_scale"), 2)
        m, v = m + (1 - BETA1) * (g - m), v + (1 - BETA2) * (g * g - v)
        w = (s["w"] if s["master"] is None else s["master"])[i].double()
        update = m / (1 - math.pow(BETA1, n)) / (torch.sqrt(v) / math.sqrt(1 - math.pow(BETA2, n)) + EPS)
        for key in ("w", "master"):
            if key in out:
                out[key][i] = w * (1 - lr * decay) - lr * update
        if c["bits"] == 8:
            out["m"][i], out["m_scale"][b] = _exact_codes(m, False)
            out["v"][i], out["v_scale"][b] = _exact_codes(torch.sqrt(v), True)
        else:
            out["m"][i], out["v"][i] = m, v
    return out


def _exact_rows(s):
    """(expert, its send rows, the rows of a they stand for)."""
    lo, c = 0, s["case"]
    for e, n in enumerate(s["counts"].tolist()):
        rows = torch.arange(lo, lo + n, device="cuda")
        from_token = s["a"].shape[0] != s["src"].numel() or c.get("gather") or c["op"] == "gate_up"
        yield e, rows, torch.div(s["src"][rows].long(), c["k"], rounding_mode="floor") if from_token else rows
        lo += n


def _matrix(w, rows, cols, c):
    """f64 [rows, cols] of one expert's packed weights, place by place."""
    r, k = torch.arange(rows, device="cuda")[:, None], torch.arange(cols, device="cuda")[None, :]
    q, per = k % BLOCK, BLOCK // c["group"]
    chunk, dword, inner = (q % 32) // 8, q // 32, q % 8
    byte, high = (inner % 4, inner // 4) if c["codes"] == "int4" else (inner // 2, inner % 2)
    place = 16 * (16 * chunk + r % 16) + 4 * dword + byte
    size = w.shape[-1]
    base = ((r // 16) * w.shape[1] + k // BLOCK) * size
    flat = w.reshape(-1)
    code = (flat[base + place] >> (4 * high).to(torch.uint8)) & 15
    value = code.double() - 8 if c["codes"] == "int4" else torch.tensor(E2M1, dtype=torch.float64, device="cuda")[code.long()]
    halves = flat.view(DTYPES[c["act"]])
    return value * halves[base // 2 + 512 + (r % 16) * per + q // c["group"]].double()


def _silu(t):
    return t / (1 + torch.exp(-t))


def exact(case, seed):
    s = prepare(case, seed)
    c, act = s["case"], DTYPES[case["act"]]
    if c["op"] == "adamw":
        return _exact_adamw(s)
    if c["op"] == "grad":
        dw = torch.zeros(c["E"], c["N"], c["K"], dtype=torch.float64, device="cuda")
        for e, rows, from_rows in _exact_rows(s):
            dw[e] = s["dy"][rows].double().t() @ s["a"][from_rows].double()
            if c["add"]:
                dw[e] += s["dw"][e]
        return {"dw": dw}
    if c["op"] in ("gate_up", "down"):
        got, n = [], 2 * c["I"] if c["op"] == "gate_up" else c["N"]
        for e, rows, from_rows in _exact_rows(s):
            z = s["a"][from_rows].double() @ _matrix(s["w"][e], n, c["K"], c).t()
            got.append(_silu(z[:, :c["I"]]) * z[:, c["I"]:] if c["op"] == "gate_up" else z)
        return {"y": torch.cat(got)}
    # the layer: one (token, slot) pair after the other, best logit first
    order = torch.argsort(-s["logits"].double(), dim=1, stable=True)[:, :c["k"]]
    gate = torch.softmax(torch.gather(s["logits"].double(), 1, order), dim=1)
    out = torch.zeros(c["T"], c["H"], dtype=torch.float64, device="cuda")
    for e in order.unique().tolist():
        t, j = torch.nonzero(order == e, as_tuple=True)
        z = s["x"][t].double() @ _matrix(s["w_up"][e], 2 * c["I"], c["H"], c).t()
        h = (_silu(z[:, :c["I"]]) * z[:, c["I"]:]).to(act).double()
        out[t] += gate[t, j].unsqueeze(1) * (h @ _matrix(s["w_down"][e], c["H"], c["I"], c).t())
    return {"idx": order.to(torch.int32), "w": gate, "out": out}
