"""Measured cases of the layer around the routing: the norm before the router
(with its residual, its 8-bit output and its gradient), the experts' products
over the routed rows in block-scaled 8-bit floating point, and the whole
layer for a few tokens.

`run` computes each operator in its plain form (elementary torch operations
in 32 bits, rounded once at the end) or, with `own` set, through the package's
entry points. `exact` gives the same outputs from the definitions in 64 bits.

8-bit rows hold e4m3 numbers and one f32 scale for each block of 128 columns;
both are returned.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
TINY = 2.0 ** -100
EPS = 1e-6
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # one decoded token between two layers: latency
        dict(name="norm_1_token", op="norm", T=1, H=4096, act="f16", residual=True, y=True, q=True),
        # a training batch in front of the router: 16-bit rows for the router, 8-bit rows for the experts
        dict(name="norm_train", op="norm", T=16384, H=4096, act="bf16", residual=True, y=True, q=True),
        # a ragged prompt whose width ends inside a scale block; first layer, no residual
        dict(name="norm_ragged_q", op="norm", T=4099, H=2872, act="f16", residual=False, y=False, q=True),
        # the same batch's backward pass, with the gradient that arrives along the residual
        dict(name="norm_backward_train", op="norm_backward", T=16384, H=4096, act="bf16", residual=True),
        # gate and up products of the top-2 batch, fused SwiGLU, 8-bit rows out
        dict(name="gate_up_top2", op="gate_up", T=16384, E=64, k=2, K=4096, I=2048, act="bf16", skew=0.0),
        # the same products of a decode batch: every expert's weights for a few rows each
        dict(name="gate_up_decode", op="gate_up", T=256, E=256, k=8, K=4096, I=2048, act="f16", skew=0.0),
        # down product of the skewed top-6 batch: segments from empty to the whole batch
        dict(name="down_top6_skewed", op="down", T=16384, E=64, k=6, K=1024, N=2048, act="bf16", skew=1.2),
        # down product of one prompt chunk of the widest workload
        dict(name="down_wide", op="down", T=8192, E=256, k=8, K=2048, N=7168, act="bf16", skew=0.0),
        # odd sizes: a width that ends inside a scale block, an odd token count
        dict(name="down_ragged", op="down", T=1021, E=8, k=2, K=1424, N=2872, act="f16", skew=0.0),
        # the whole layer for one decoded token
        dict(name="layer_1_token", op="layer", T=1, E=256, k=8, H=4096, I=2048, act="f16", weights="e4m3"),
        # the whole layer for a small batch with 16-bit weights
        dict(name="layer_8_tokens_16bit", op="layer", T=8, E=64, k=2, H=4096, I=2048, act="bf16", weights="16"),
        # the whole layer for a decode batch of the widest workload
        dict(name="layer_32_tokens_wide", op="layer", T=32, E=256, k=8, H=7168, I=2048, act="bf16", weights="e4m3"),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "gate_up", "down", "layer"])
    act = rng.choice(["f16", "bf16"])
    if op in ("norm", "norm_backward"):
        H = _log(rng, 128, 8192, 8)
        T = _log(rng, 1, min(32768, 16384 * 4096 // H))
        c = dict(op=op, T=T, H=H, act=act, residual=rng.random() < 0.7)
        if op == "norm":
            c["q"] = rng.random() < 0.75
            c["y"] = not c["q"] or rng.random() < 0.6
        return c
    if op == "layer":
        E = rng.choice([8, 16, 64, 160, 256])
        return dict(op=op, T=rng.randint(1, 64 if E <= 64 else 32), E=E, k=rng.randint(1, 8),
                    H=_log(rng, 512, 4096, 16), I=_log(rng, 128, 2048, 16), act=act,
                    weights=rng.choice(["e4m3", "e4m3", "16"]))
    E = rng.choice([4, 8, 32, 64, 160, 256])
    k = rng.randint(1, min(E, 8))
    K = _log(rng, 256, 7168, 16)
    skew = rng.choice([0.0, 0.0, 1.2]) if E <= 64 else 0.0
    c = dict(op=op, E=E, k=k, K=K, act=act, skew=skew)
    if op == "gate_up":
        c["I"] = _log(rng, 128, 2048, 16)
        width = 2 * c["I"]
    else:
        c["N"] = _log(rng, 256, 7168, 8)
        width = c["N"]
    most = 10 ** 12 // (k * K * width)  # at most 2e12 operations
    c["T"] = _log(rng, 1, max(1, min(16384, most)))
    return c


# ---- inputs ----------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _codes(shape, g):
    """e4m3 codes of normal values, as a quantised weight or activation has."""
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    for part in out.view(-1).split(1 << 28):
        part.copy_((torch.randn(part.shape, dtype=torch.bfloat16, device="cuda", generator=g) * 110).clamp_(-448, 448))
    return out


def _scales(shape, size, g):
    """f32 scales around `size`, spread over about a factor of three."""
    return (torch.rand(shape, device="cuda", generator=g) + 0.5) * size


def _blocks(n):
    return -(-n // BLOCK)


def _logits(T, E, skew, g):
    """Router logits; with a skew the experts' popularity falls as a power of their (shuffled) rank."""
    logits = torch.randn(T, E, device="cuda", generator=g)
    if skew:
        rank = torch.randperm(E, device="cuda", generator=g).float() + 1
        logits = logits - skew * torch.log(rank)
    return logits


def prepare(case, seed):
    g, c = _gen(seed), dict(case)
    op, act = c["op"], DTYPES[c["act"]]
    rand = lambda *s: torch.randn(s, device="cuda", generator=g).to(act)  # noqa: E731
    s = {"case": c}
    if op in ("norm", "norm_backward"):
        T, H = c["T"], c["H"]
        s["x"] = rand(T, H)
        s["residual"] = rand(T, H) * 2 if c["residual"] else None
        s["gamma"] = (1 + 0.2 * torch.randn(H, device="cuda", generator=g)).to(act)
        if op == "norm_backward":
            # the forward pass kept its residual stream and 1 / rms
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
            s["dy"] = rand(T, H)
        return s
    if op == "layer":
        T, E, H, I = c["T"], c["E"], c["H"], c["I"]
        s["logits"] = _logits(T, E, 0.0, g)
        s["x"] = rand(T, H)
        for name, rows, cols in (("up", 2 * I, H), ("down", H, I)):
            if c["weights"] == "e4m3":
                s["w_" + name] = _codes((E, rows, cols), g)
                s["s_" + name] = _scales((E, _blocks(rows), _blocks(cols)), 1 / (110 * math.sqrt(cols)), g)
            else:
                s["w_" + name] = torch.randn(E, rows, cols, dtype=act, device="cuda", generator=g) / math.sqrt(cols)
                s["s_" + name] = None
        return s
    T, E, k, K = c["T"], c["E"], c["k"], c["K"]
    # the routed batch, as the layout gives it: rows by expert, then by token
    idx = torch.sort(_logits(T, E, c["skew"], g), dim=1, descending=True, stable=True)[1][:, :k]
    s["src"] = torch.argsort(idx.reshape(-1), stable=True).to(torch.int32)
    counts = torch.bincount(idx.reshape(-1), minlength=E)
    s["counts"] = counts.to(torch.int32)
    s["offsets"] = (torch.cumsum(counts, 0) - counts).to(torch.int32)
    rows, N = (T, 2 * c["I"]) if op == "gate_up" else (T * k, c["N"])
    s["a"] = _codes((rows, K), g)
    s["a_scale"] = _scales((rows, _blocks(K)), 1 / 110, g)
    s["b"] = _codes((E, N, K), g)
    s["b_scale"] = _scales((E, _blocks(N), _blocks(K)), 1 / (110 * math.sqrt(K)), g)
    return s


# ---- the plain form ----------------------------------------------------------

def _quantise(v):
    """8-bit rows of f32 v: (e4m3 numbers, scales)."""
    rows, cols = v.shape
    nb = _blocks(cols)
    p = torch.zeros(rows, nb * BLOCK, device=v.device)
    p[:, :cols] = v
    p = p.view(rows, nb, BLOCK)
    scale = p.abs().amax(2).clamp_min(TINY) / E4M3_MAX
    code = (p / scale[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return code.view(rows, -1)[:, :cols].contiguous(), scale


def _wide(scale, cols):
    return scale.repeat_interleave(BLOCK, dim=-1)[..., :cols]


def _weights(w, scale):
    if scale is None:
        return w.float()
    f = w.float()
    f *= _wide(scale, w.shape[-1]).repeat_interleave(BLOCK, dim=-2)[..., :w.shape[-2], :]
    return f


def _plain_norm(s):
    c = s["case"]
    v = s["x"].float()
    out = {}
    if c["residual"]:
        out["h"] = (v + s["residual"].float()).to(s["x"].dtype)
        v = out["h"].float()
    out["rstd"] = torch.rsqrt(v.square().mean(1) + EPS)
    v = v * out["rstd"][:, None] * s["gamma"].float()
    if c["y"]:
        out["y"] = v.to(s["x"].dtype)
    if c["q"]:
        out["q"], out["scale"] = _quantise(v)
    return out


def _plain_norm_backward(s):
    n = s["x"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    t = dy * s["gamma"].float()
    dx = s["rstd"][:, None] * (t - n * (t * n).mean(1, keepdim=True))
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    return {"dx": dx.to(s["x"].dtype), "dgamma": (dy * n).sum(0)}


def _plain_product(s, gather):
    """Rows of every expert padded to the longest segment, one batched product."""
    c = s["case"]
    rows = torch.arange(s["src"].numel(), device="cuda")
    expert = torch.repeat_interleave(torch.arange(c["E"], device="cuda"), s["counts"].long())
    place = rows - s["offsets"].long()[expert]
    a = s["a"].float() * _wide(s["a_scale"], c["K"])
    if gather:
        a = a[s["src"].long() // c["k"]]
    padded = torch.zeros(c["E"], int(s["counts"].max()), c["K"], device="cuda")
    padded[expert, place] = a
    w = _weights(s["b"], s["b_scale"])
    return torch.bmm(padded, w.transpose(1, 2))[expert, place]


def _plain_layer(s):
    c = s["case"]
    top, idx = torch.sort(s["logits"], dim=1, descending=True, stable=True)
    top, idx = top[:, :c["k"]].double(), idx[:, :c["k"]]
    e = torch.exp(top - top[:, :1])
    w = (e / e.sum(1, keepdim=True)).float()
    pick = idx.reshape(-1)
    scale = lambda n: None if s[n] is None else s[n][pick]  # noqa: E731
    x = s["x"].float().repeat_interleave(c["k"], dim=0)[:, :, None]
    z = torch.bmm(_weights(s["w_up"][pick], scale("s_up")), x)[:, :, 0]
    gate, up = z[:, :c["I"]], z[:, c["I"]:]
    h = (gate * torch.sigmoid(gate) * up).to(s["x"].dtype).float()
    y = torch.bmm(_weights(s["w_down"][pick], scale("s_down")), h[:, :, None])[:, :, 0]
    out = (y.view(c["T"], c["k"], -1) * w[:, :, None]).sum(1)
    return {"idx": idx.to(torch.int32), "w": w, "out": out.to(s["x"].dtype)}


def _plain(s):
    op = s["case"]["op"]
    if op == "norm":
        return _plain_norm(s)
    if op == "norm_backward":
        return _plain_norm_backward(s)
    if op == "layer":
        return _plain_layer(s)
    z = _plain_product(s, gather=op == "gate_up")
    if op == "down":
        return {"y": z.to(DTYPES[s["case"]["act"]])}
    gate, up = z[:, :s["case"]["I"]], z[:, s["case"]["I"]:]
    q, scale = _quantise(gate * torch.sigmoid(gate) * up)
    return {"q": q, "scale": scale}


# ---- the package's calls -----------------------------------------------------

def _own(s):
    from combine_router_topk_amd import binding as B
    c = s["case"]
    act = DTYPES[c["act"]]
    fmt = B.MOE_F16 if c["act"] == "f16" else B.MOE_BF16
    new = lambda *shape, dtype=act: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
    f32, e4m3 = torch.float32, torch.float8_e4m3fn
    if c["op"] in ("norm", "norm_backward"):
        T, H = c["T"], c["H"]
        p = B.make_problem(T, 1, 1, H, 1, fmt)
        if c["op"] == "norm_backward":
            dx, dgamma = new(T, H), new(H, dtype=f32)
            ws = new(B.moe_rms_norm_workspace_bytes(p), dtype=torch.uint8)
            B.moe_rms_norm_backward(p, s["dy"], s["residual"], s["x"], s["gamma"], s["rstd"], dx, dgamma, ws)
            return {"dx": dx, "dgamma": dgamma}
        out = {"rstd": new(T, dtype=f32)}
        if c["residual"]:
            out["h"] = new(T, H)
        if c["y"]:
            out["y"] = new(T, H)
        if c["q"]:
            out["q"], out["scale"] = new(T, H, dtype=e4m3), new(T, _blocks(H), dtype=f32)
        B.moe_rms_norm(p, s["x"], s["residual"], s["gamma"], EPS, out.get("h"), out.get("y"), out.get("q"),
                       out.get("scale"), out["rstd"])
        return out
    T, E, k = c["T"], c["E"], c["k"]
    if c["op"] == "layer":
        p = B.make_problem(T, E, k, c["H"], 1, fmt)
        idx, w, out = new(T, k, dtype=torch.int32), new(T, k, dtype=f32), new(T, c["H"])
        ws = new(B.moe_layer_workspace_bytes(p, c["I"]), dtype=torch.uint8)
        B.moe_layer_few_tokens(p, c["I"], s["logits"], s["x"], s["w_up"], s["s_up"], s["w_down"], s["s_down"],
                               idx, w, out, ws)
        return {"idx": idx, "w": w, "out": out}
    p = B.make_problem(T, E, k, c["K"], 1, fmt)
    if c["op"] == "down":
        y = new(T * k, c["N"])
        B.moe_expert_gemm(p, c["K"], c["N"], s["a"], s["a_scale"], None, s["b"], s["b_scale"], s["counts"],
                          s["offsets"], y)
        return {"y": y}
    q, scale = new(T * k, c["I"], dtype=e4m3), new(T * k, _blocks(c["I"]), dtype=f32)
    B.moe_expert_gemm_swiglu(p, c["K"], c["I"], s["a"], s["a_scale"], s["src"], s["b"], s["b_scale"],
                             s["counts"], s["offsets"], q, scale)
    return {"q": q, "scale": scale}


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ---- what a pass cannot do without -------------------------------------------

def work(case):
    c = case
    if c["op"] == "norm":
        per = 2 + (4 if c["residual"] else 0) + (2 if c["y"] else 0)
        n = c["T"] * c["H"]
        q = n + 4 * c["T"] * _blocks(c["H"]) if c["q"] else 0
        return {"bytes": per * n + q + 2 * c["H"] + 4 * c["T"], "flops": 6 * n}
    if c["op"] == "norm_backward":
        n = c["T"] * c["H"]
        return {"bytes": (8 if c["residual"] else 6) * n + 4 * c["T"] + 6 * c["H"], "flops": 10 * n}
    T, E, k = c["T"], c["E"], c["k"]
    active = min(E, T * k, max(k, round(E * (1 - (1 - k / E) ** T))))
    if c["op"] == "layer":
        weights = 3 * c["H"] * c["I"]
        per = 1 + 4 / BLOCK ** 2 if c["weights"] == "e4m3" else 2
        return {"bytes": int(active * weights * per) + 4 * T * E + 4 * T * c["H"] + 8 * T * k,
                "flops": 2 * T * k * weights}
    rows = T * k
    if c["op"] == "down":
        K, N = c["K"], c["N"]
        other = rows * (K + 4 * _blocks(K)) + 2 * rows * N
    else:
        K, N = c["K"], 2 * c["I"]
        other = T * (K + 4 * _blocks(K)) + rows * (c["I"] + 4 * _blocks(c["I"]))
    return {"bytes": active * (N * K + 4 * _blocks(N) * _blocks(K)) + other + 8 * E + 4 * rows,
            "flops": 2 * rows * K * N}


# ---- the definitions in 64 bits ------------------------------------------------

def _exact_rows(v):
    """8-bit rows of f64 v, block by block: (numbers, scales)."""
    numbers, scales = torch.empty_like(v), []
    for lo in range(0, v.shape[1], BLOCK):
        part = v[:, lo:lo + BLOCK]
        scale = torch.clamp(part.abs().max(dim=1, keepdim=True).values, min=TINY) / 448
        t = part / scale
        # spacing of e4m3 around t: 2^-3 of its power of two, 2^-9 below 2^-6
        step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
        numbers[:, lo:lo + BLOCK] = torch.clamp(torch.round(t / step) * step, -448, 448)
        scales.append(scale)
    return numbers, torch.cat(scales, 1)


def _spread(scale, shape):
    """A block's scale at each place of the matrix it covers."""
    i = torch.arange(shape[-2], device=scale.device) // BLOCK
    j = torch.arange(shape[-1], device=scale.device) // BLOCK
    return scale.double()[i][:, j]


def _matrix(w, scale):
    return w.double() if scale is None else w.double() * _spread(scale, w.shape)


def _exact_product(s, finish):
    c = s["case"]
    a_all, at = s["a"], torch.arange(c["K"], device="cuda") // BLOCK
    got, lo = [], 0
    for e, n in enumerate(s["counts"].tolist()):
        if not n:
            continue
        rows = torch.arange(lo, lo + n, device="cuda")
        if c["op"] == "gate_up":
            rows = torch.div(s["src"][rows].long(), c["k"], rounding_mode="floor")
        a = a_all[rows].double() * s["a_scale"][rows].double()[:, at]
        got.append(finish(a @ _matrix(s["b"][e], s["b_scale"][e]).t()))
        lo += n
    return got


def _silu(t):
    return t / (1 + torch.exp(-t))


def exact(case, seed):
    s = prepare(case, seed)
    c, act = s["case"], DTYPES[case["act"]]
    if c["op"] == "norm":
        h, out = s["x"].double(), {}
        if c["residual"]:
            out["h"] = (h + s["residual"].double()).to(act).double()
            h = out["h"]
        out["rstd"] = 1 / torch.sqrt((h * h).sum(1) / c["H"] + EPS)
        v = s["gamma"].double() * (h * out["rstd"].unsqueeze(1))
        if c["y"]:
            out["y"] = v
        if c["q"]:
            out["q"], out["scale"] = _exact_rows(v)
        return out
    if c["op"] == "norm_backward":
        r, dy = s["rstd"].double().unsqueeze(1), s["dy"].double()
        n, g = s["x"].double() * r, s["gamma"].double()
        dot = (dy * g * n).sum(1, keepdim=True) / c["H"]
        dx = r * dy * g - r * n * dot
        if c["residual"]:
            dx += s["residual"].double()
        return {"dx": dx, "dgamma": (dy * n).sum(0)}
    if c["op"] == "down":
        return {"y": torch.cat(_exact_product(s, lambda z: z))}
    if c["op"] == "gate_up":
        parts = _exact_product(s, lambda z: _exact_rows(_silu(z[:, :c["I"]]) * z[:, c["I"]:]))
        return {"q": torch.cat([p[0] for p in parts]), "scale": torch.cat([p[1] for p in parts])}
    # the layer: one (token, slot) pair after the other, best logit first
    order = torch.argsort(-s["logits"].double(), dim=1, stable=True)[:, :c["k"]]
    gate = torch.softmax(torch.gather(s["logits"].double(), 1, order), dim=1)
    out = torch.zeros(c["T"], c["H"], dtype=torch.float64, device="cuda")
    for e in order.unique().tolist():
        t, j = torch.nonzero(order == e, as_tuple=True)
        up = _matrix(s["w_up"][e], None if s["s_up"] is None else s["s_up"][e])
        down = _matrix(s["w_down"][e], None if s["s_down"] is None else s["s_down"][e])
        z = s["x"][t].double() @ up.t()
        h = (_silu(z[:, :c["I"]]) * z[:, c["I"]:]).to(act).double()
        out[t] += gate[t, j].unsqueeze(1) * (h @ down.t())
    return {"idx": order.to(torch.int32), "w": gate, "out": out}
