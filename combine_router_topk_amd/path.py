"""The whole routing path on device buffers: route -> greedy replica
assignment -> layout -> dispatch -> expert stand-in -> combine, each step one
call into the HIP library. Torch provides the device memory and the stream.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import binding as B


@dataclass
class Buffers:
    p: B.Problem
    logits: torch.Tensor
    x: torch.Tensor
    rep: torch.Tensor | None
    maxrep: int
    ws: torch.Tensor
    idx: torch.Tensor
    w: torch.Tensor
    counts: torch.Tensor
    assign: torch.Tensor
    active: torch.Tensor
    rank_of: torch.Tensor
    expert_offsets: torch.Tensor
    rank_offsets: torch.Tensor
    pos: torch.Tensor
    src: torch.Tensor
    dedup: torch.Tensor
    send: torch.Tensor
    y: torch.Tensor
    out: torch.Tensor


def allocate(p: B.Problem, logits: torch.Tensor, x: torch.Tensor, rep: torch.Tensor | None = None,
             device: str | torch.device = "cuda") -> Buffers:
    """Device buffers for one batch. `logits` [T, E] f32 and `x` [T, H] in the
    activation dtype are copied to the device; `rep` is an int32 [E, maxrep]
    replica table or None."""
    dev = torch.device(device)
    T, E, k, H, R = p.T, p.E, p.k, p.H, p.R
    act = B._TORCH_ACT[p.act_dtype]
    i32 = dict(dtype=torch.int32, device=dev)
    out_dt = torch.float32 if p.flags & B.MOE_FLAG_OUT_F32 else act
    rep_d = None if rep is None else rep.to(dev, torch.int32).contiguous()
    maxrep = 1 if rep is None else int(rep.shape[1])
    ws_bytes = B.moe_workspace_bytes(p)
    return Buffers(
        p=p, logits=logits.to(dev, torch.float32).contiguous(), x=x.to(dev).contiguous(),
        rep=rep_d, maxrep=maxrep,
        ws=torch.empty(ws_bytes, dtype=torch.uint8, device=dev),
        idx=torch.empty(T * k, **i32), w=torch.empty(T * k, dtype=torch.float32, device=dev),
        counts=torch.empty(E, **i32), assign=torch.empty(E, **i32), active=torch.empty(R, **i32),
        rank_of=torch.empty(E, **i32), expert_offsets=torch.empty(E, **i32),
        rank_offsets=torch.empty(R + 1, **i32), pos=torch.empty(T * k, **i32),
        src=torch.empty(T * k, **i32), dedup=torch.empty(R, **i32),
        send=torch.empty(T * k, H, dtype=act, device=dev),
        y=torch.empty(T * k, H, dtype=act, device=dev),
        out=torch.empty(T, H, dtype=out_dt, device=dev))


def route(b: Buffers, stream=None) -> None:
    B.moe_route(b.p, b.logits, b.idx, b.w, b.counts, b.ws, stream)


def assign(b: Buffers, stream=None) -> None:
    B.moe_assign_replicas(b.p, b.counts, b.rep, b.maxrep, b.assign, b.active, stream)


def layout(b: Buffers, stream=None) -> None:
    B.moe_layout(b.p, b.idx, b.assign, b.rep, b.maxrep, b.rank_of, b.expert_offsets,
                 b.rank_offsets, b.pos, b.src, b.dedup, b.ws, stream)


def route_assign_layout(b: Buffers, stream=None) -> None:
    """route, assign and layout in one library call (two launches for a
    decode-sized batch)."""
    B.moe_route_assign_layout(b.p, b.logits, b.rep, b.maxrep, b.idx, b.w, b.counts, b.assign,
                              b.active, b.rank_of, b.expert_offsets, b.rank_offsets, b.pos, b.src,
                              b.dedup, b.ws, stream)


def dispatch(b: Buffers, stream=None) -> None:
    B.moe_dispatch(b.p, b.x, b.pos, b.send, stream)


def standin(b: Buffers, stream=None) -> None:
    B.moe_expert_standin(b.p, b.send, b.src, b.idx, b.y, stream)


def combine(b: Buffers, stream=None) -> None:
    B.moe_combine(b.p, b.y, b.pos, b.w, b.out, stream)


STEPS = (route, assign, layout, dispatch, standin, combine)
# the same pass with route, assign and layout in one call
FUSED_STEPS = (route_assign_layout, dispatch, standin, combine)


def run(b: Buffers, stream=None) -> None:
    for step in STEPS:
        step(b, stream)


def capture(b: Buffers, steps=STEPS) -> torch.cuda.CUDAGraph:
    """Records one pass of `steps` (the whole path by default) into a HIP
    graph. The library only enqueues kernels (no memset, allocation or
    synchronisation), so the pass replays with one launch; the buffers of `b`
    are the graph's inputs and outputs: copy a new batch into b.logits / b.x
    in place, then replay. One eager pass on a side stream comes first, as
    torch asks before a capture."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for step in steps:
            step(b)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for step in steps:
            step(b)
    return g


def record(b: Buffers, ss: SingleSend | None = None) -> dict:
    """Host-side record of one routed batch: what "METRO AllGather vs AllToAll
    for MoE decode", section "Distinguish METRO from backend names", asks to
    keep beside collective traces (buffer sizes per destination rank and the
    expert replica chosen for each expert's global count), plus the dedup
    total and the activated experts per GPU. Reads back 2E + 3R + 1 ints of
    metadata (R + 1 more with `ss`; this synchronises the stream), never the
    rows.

    send_bytes[r] is rank r's segment of the send buffer, the size of the
    all-to-all chunk for destination r; with `ss`, ss_send_bytes[r] is the
    same for the single-send buffer."""
    p = b.p
    row_bytes = p.H * 2  # 16-bit activations
    roff = b.rank_offsets.cpu().tolist()
    rec = {
        "T": p.T, "E": p.E, "k": p.k, "H": p.H, "R": p.R,
        "send_bytes": [(roff[r + 1] - roff[r]) * row_bytes for r in range(p.R)],
        "rows": roff[-1],
        "dedup_rows": int(b.dedup.sum().item()),
        "active_per_gpu": b.active.cpu().tolist(),
        "counts": b.counts.cpu().tolist(),
        "assign": b.assign.cpu().tolist(),
    }
    if ss is not None:
        so = ss.ss_rank_offsets.cpu().tolist()
        rec["ss_send_bytes"] = [(so[r + 1] - so[r]) * row_bytes for r in range(p.R)]
    return rec


@dataclass
class SingleSend:
    """Single-send buffers: one row per (token, destination rank). The row
    capacity is T * min(k, R), the most distinct (token, rank) pairs a batch
    can have, so no count has to be read back before the dispatch."""
    ss_rank_offsets: torch.Tensor
    ss_row: torch.Tensor
    ss_token: torch.Tensor
    send_ss: torch.Tensor


def allocate_single_send(b: Buffers) -> SingleSend:
    p, dev = b.p, b.idx.device
    n, cap = p.T * p.k, p.T * min(p.k, p.R)
    i32 = dict(dtype=torch.int32, device=dev)
    return SingleSend(ss_rank_offsets=torch.empty(p.R + 1, **i32), ss_row=torch.empty(n, **i32),
                      ss_token=torch.empty(n, **i32),
                      send_ss=torch.empty(cap, p.H, dtype=b.send.dtype, device=dev))


def layout_single_send(b: Buffers, ss: SingleSend, stream=None) -> None:
    B.moe_layout_single_send(b.p, b.idx, b.assign, b.rep, b.maxrep, b.rank_of, b.expert_offsets,
                             b.rank_offsets, b.pos, b.src, b.dedup, ss.ss_rank_offsets, ss.ss_row,
                             ss.ss_token, b.ws, stream)


def route_assign_layout_single_send(b: Buffers, ss: SingleSend, stream=None) -> None:
    """route, assign and the single-send layout in one library call (three
    launches for a batch without a replica table)."""
    B.moe_route_assign_layout_single_send(b.p, b.logits, b.rep, b.maxrep, b.idx, b.w, b.counts,
                                          b.assign, b.active, b.rank_of, b.expert_offsets,
                                          b.rank_offsets, b.pos, b.src, b.dedup,
                                          ss.ss_rank_offsets, ss.ss_row, ss.ss_token, b.ws, stream)


def single_send_dispatch(b: Buffers, ss: SingleSend, stream=None) -> None:
    B.moe_single_send_dispatch(b.p, b.x, ss.ss_row, ss.send_ss, stream)


def single_send_expand(b: Buffers, ss: SingleSend, stream=None) -> None:
    """Fills b.send from the single-send rows (what dispatch writes)."""
    B.moe_single_send_expand(b.p, ss.send_ss, ss.ss_rank_offsets, ss.ss_token, ss.ss_row, b.pos,
                             b.send, stream)


@dataclass
class Stats:
    """Routing-statistics outputs: send_counts [R, R], coselect [E, E] (or
    None), stats [4] = max/mean, Gini, Dirichlet alpha, locality."""
    send_counts: torch.Tensor
    coselect: torch.Tensor | None
    stats: torch.Tensor


def allocate_stats(b: Buffers, coselect: bool = True) -> Stats:
    p, dev = b.p, b.idx.device
    return Stats(send_counts=torch.empty(p.R, p.R, dtype=torch.int32, device=dev),
                 coselect=torch.empty(p.E, p.E, dtype=torch.int32, device=dev) if coselect else None,
                 stats=torch.empty(4, dtype=torch.float64, device=dev))


def routing_stats(b: Buffers, st: Stats, stream=None) -> None:
    B.moe_routing_stats(b.p, b.idx, b.counts, b.rank_of, st.send_counts, st.coselect, st.stats,
                        stream)


@dataclass
class Split:
    """Token-balanced (EPLB-style) routing outputs: the GPU of each pair and,
    per GPU, the activated replicas and the pairs served."""
    gpu_of_pair: torch.Tensor
    active: torch.Tensor
    tokens: torch.Tensor


def allocate_split(b: Buffers) -> Split:
    p, dev = b.p, b.idx.device
    i32 = dict(dtype=torch.int32, device=dev)
    return Split(gpu_of_pair=torch.empty(p.T * p.k, **i32), active=torch.empty(p.R, **i32),
                 tokens=torch.empty(p.R, **i32))


def token_balanced_split(b: Buffers, sp: Split, stream=None) -> None:
    B.moe_token_balanced_split(b.p, b.idx, b.counts, b.pos, b.expert_offsets, b.rep, b.maxrep,
                               sp.gpu_of_pair, sp.active, sp.tokens, stream)


@dataclass
class ExpertWeights:
    """The experts' weights in 8 bits: w_up [E, 2 I, H] (gate rows first) and
    w_down [E, H, I] in float8_e4m3fn, with one fp32 scale for each block of
    128 x 128 (s_up, s_down); or both in the activation format without scales,
    for the layer of a few tokens."""
    I: int
    w_up: torch.Tensor
    s_up: torch.Tensor | None
    w_down: torch.Tensor
    s_down: torch.Tensor | None


@dataclass
class Layer:
    """Buffers of the layer around the routing: the normed token rows in 8
    bits, the experts' inner rows in 8 bits, 1 / rms of each token."""
    I: int
    xq: torch.Tensor
    xq_scale: torch.Tensor
    rstd: torch.Tensor
    hq: torch.Tensor
    hq_scale: torch.Tensor


def allocate_layer(b: Buffers, I: int) -> Layer:
    p, dev = b.p, b.idx.device
    n, f32 = p.T * p.k, dict(dtype=torch.float32, device=dev)
    return Layer(I=I, xq=torch.empty(p.T, p.H, dtype=B.E4M3, device=dev),
                 xq_scale=torch.empty(p.T, B.scale_blocks(p.H), **f32),
                 rstd=torch.empty(p.T, **f32), hq=torch.empty(n, I, dtype=B.E4M3, device=dev),
                 hq_scale=torch.empty(n, B.scale_blocks(I), **f32))


def norm(b: Buffers, l: Layer, x: torch.Tensor, residual: torch.Tensor | None, gamma: torch.Tensor,
         eps: float = 1e-6, h: torch.Tensor | None = None, stream=None) -> None:
    """The rows the router scores (b.x) and the experts take (l.xq) from the
    layer's input x and the residual stream, which becomes h."""
    B.moe_rms_norm(b.p, x, residual, gamma, eps, h, b.x, l.xq, l.xq_scale, l.rstd, stream)


def expert_gate_up(b: Buffers, l: Layer, w: ExpertWeights, stream=None) -> None:
    """The experts' inner rows, straight from the token rows (no dispatch)."""
    B.moe_expert_gemm_swiglu(b.p, b.p.H, l.I, l.xq, l.xq_scale, b.src, w.w_up, w.s_up, b.counts,
                             b.expert_offsets, l.hq, l.hq_scale, stream)


def _act_out(p: B.Problem) -> B.Problem:
    """The problem with rows in the activation format, whatever b.out is in."""
    return p if not p.flags & B.MOE_FLAG_OUT_F32 else \
        B.make_problem(p.T, p.E, p.k, p.H, p.R, p.act_dtype, p.flags & ~B.MOE_FLAG_OUT_F32)


def expert_down(b: Buffers, l: Layer, w: ExpertWeights, stream=None) -> None:
    """The experts' outputs in send order (what standin writes otherwise); bf16
    rows from exact sums if the problem has MOE_FLAG_EXACT_SUMS."""
    p = _act_out(b.p)
    B.moe_expert_gemm(p, l.I, p.H, l.hq, l.hq_scale, None, w.w_down, w.s_down, b.counts,
                      b.expert_offsets, b.y, stream)


def run_layer(b: Buffers, l: Layer, w: ExpertWeights, stream=None) -> None:
    """Routing, the experts' products and the combine, from b.logits and l's
    8-bit rows to b.out."""
    route_assign_layout(b, stream)
    expert_gate_up(b, l, w, stream)
    expert_down(b, l, w, stream)
    combine(b, stream)


def layer_few_tokens(b: Buffers, w: ExpertWeights, ws: torch.Tensor, stream=None) -> None:
    """The same layer for a few tokens in two to four launches, from b.logits and the
    16-bit rows b.x to b.out; `ws` has layer_workspace(b, I) bytes."""
    B.moe_layer_few_tokens(b.p, w.I, b.logits, b.x, w.w_up, w.s_up, w.w_down, w.s_down, b.idx, b.w,
                           b.out, ws, stream)


def layer_workspace(b: Buffers, I: int) -> torch.Tensor:
    return torch.empty(B.moe_layer_workspace_bytes(b.p, I), dtype=torch.uint8, device=b.idx.device)


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _packed_places(f: B.PackedFormat, device) -> tuple[torch.Tensor, torch.Tensor]:
    """Of each column of a tile, the place of its code in a row's 32 nibbles of
    each of the four chunks: (chunk, nibble)."""
    c = torch.arange(128, device=device)
    j, g, i = c // 32, c % 32 // 8, c % 8
    inner = 2 * (i % 4) + i // 4 if f.codes == B.MOE_PACKED_INT else i
    return g, 8 * j + inner


def _check_format(f: B.PackedFormat) -> None:
    if f.codes not in (B.MOE_PACKED_INT, B.MOE_PACKED_E2M1) or f.group not in (32, 64, 128) \
            or f.scale_dtype not in B._TORCH_ACT:
        raise ValueError(f"{f}: a format has integers or e2m1, groups of 32, 64 or 128 columns and 16-bit scales")


def _lay_out(q: torch.Tensor, scale: torch.Tensor, f: B.PackedFormat) -> torch.Tensor:
    """One matrix's tiles from the codes 0 .. 15 and the 16-bit scales of whole tiles' rows."""
    nt, kt, per = q.shape[0] // 16, q.shape[1] // 128, 128 // f.group
    q = q.view(nt, 16, kt, 128).to(torch.uint8)
    g, nibble = _packed_places(f, q.device)
    codes = torch.zeros(nt, kt, 4, 16, 32, dtype=torch.uint8, device=q.device)
    codes[:, :, g, :, nibble] = q.permute(3, 0, 2, 1)
    codes = codes[..., ::2] | codes[..., 1::2] << 4
    scale = scale.view(nt, 16, kt, per).transpose(1, 2).contiguous()
    return torch.cat([codes.reshape(nt, kt, 1024), scale.view(torch.uint8).view(nt, kt, -1)], 2).view(-1)


def pack_weights(w: torch.Tensor, f: B.PackedFormat) -> torch.Tensor:
    """Weights [..., rows, cols] in 4 bits (see include/moe_route.h), each group of
    columns with the scale that takes its largest magnitude to the largest code (7
    or 6), each value to the nearest code (ties to the even one). Done once for a
    model, in torch operations on w's device; returns uint8 [..., bytes]. Weights that
    are in 4 bits already keep their codes and scales with pack_codes."""
    _check_format(f)
    if w.dim() < 2 or 0 in w.shape[-2:]:
        raise ValueError("weights [..., rows, cols], one row and column at least")
    lead, (rows, cols) = w.shape[:-2], w.shape[-2:]
    nt, kt, per = -(-rows // 16), -(-cols // 128), 128 // f.group
    ints = f.codes == B.MOE_PACKED_INT
    out = []
    for m in w.reshape(-1, rows, cols):  # one matrix at a time: the fp32 copy is eight times the result
        v = torch.zeros(nt * 16, kt * 128, device=w.device)
        v[:rows, :cols] = m.float()
        if not bool(torch.isfinite(v).all()):
            raise ValueError("weights that are not finite have no 4-bit form")
        v = v.view(nt * 16, kt * per, f.group)
        scale = (v.abs().amax(2) / (7.0 if ints else 6.0)).to(B._TORCH_ACT[f.scale_dtype])
        if not bool(torch.isfinite(scale).all()):
            raise ValueError("a group's scale is beyond its 16-bit format")
        t = v / torch.where(scale == 0, 1.0, scale.float())[:, :, None]
        if ints:
            q = t.round().clamp_(-8, 7).add_(8)
        else:
            borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
            a = t.abs()  # at a border the even code: below the even borders, above the odd ones
            q = (a > borders[0]).float()
            for n, b in enumerate(borders[1:].tolist(), 1):
                q += (a >= b) if n % 2 else (a > b)
            q += 8.0 * (t < 0)
        out.append(_lay_out(q.view(nt * 16, kt * 128), scale, f))
    if not out:
        return torch.zeros(*lead, B.moe_packed_weight_bytes(f, 1, rows, cols), dtype=torch.uint8, device=w.device)
    return torch.stack(out).view(*lead, -1)


def pack_codes(codes: torch.Tensor, scale: torch.Tensor, f: B.PackedFormat) -> torch.Tensor:
    """Weights that are in 4 bits already, laid out with the codes and scales that they
    have: codes [..., rows, cols] of any whole-number type, -8 .. 7 for integers or
    the e2m1 patterns 0 .. 15, and scale [..., rows, ceil(cols / group)] in the
    format's 16 bits, the first of each row for its first `group` columns. Returns
    uint8 [..., bytes], as pack_weights does."""
    _check_format(f)
    if codes.dim() < 2 or 0 in codes.shape[-2:]:
        raise ValueError("codes [..., rows, cols], one row and column at least")
    if codes.dtype.is_floating_point or codes.dtype.is_complex or codes.dtype == torch.bool:
        raise ValueError(f"codes: dtype {codes.dtype}, expected whole numbers")
    lead, (rows, cols) = codes.shape[:-2], codes.shape[-2:]
    groups = -(-cols // f.group)
    if tuple(scale.shape) != (*lead, rows, groups) or scale.dtype != B._TORCH_ACT[f.scale_dtype]:
        raise ValueError(f"scale: {list(scale.shape)} {scale.dtype}, codes {list(codes.shape)} in groups of {f.group} "
                         f"need {[*lead, rows, groups]} {B._TORCH_ACT[f.scale_dtype]}")
    nt, kt, per = -(-rows // 16), -(-cols // 128), 128 // f.group
    zero = 8 if f.codes == B.MOE_PACKED_INT else 0
    out = []
    for c, s in zip(codes.reshape(-1, rows, cols), scale.reshape(-1, rows, groups)):
        lo, hi = (int(x) for x in c.aminmax())
        if lo < -zero or hi > 15 - zero:
            raise ValueError(f"codes outside {-zero} .. {15 - zero}")
        if not bool(torch.isfinite(s).all()):
            raise ValueError("a group's scale is not finite")
        q = torch.full((nt * 16, kt * 128), zero, dtype=torch.uint8, device=codes.device)
        q[:rows, :cols] = (c.to(torch.int16) + zero).to(torch.uint8)
        whole = torch.zeros(nt * 16, kt * per, dtype=s.dtype, device=codes.device)
        whole[:rows, :groups] = s
        out.append(_lay_out(q, whole, f))
    if not out:
        return torch.zeros(*lead, B.moe_packed_weight_bytes(f, 1, rows, cols), dtype=torch.uint8, device=codes.device)
    return torch.stack(out).view(*lead, -1)


def unpack_weights(packed: torch.Tensor, rows: int, cols: int, f: B.PackedFormat) -> torch.Tensor:
    """The fp32 values [..., rows, cols] that packed weights stand for."""
    _check_format(f)
    if packed.dtype != torch.uint8 or rows < 1 or cols < 1 or packed.shape[-1] != B.moe_packed_weight_bytes(f, 1, rows, cols):
        raise ValueError(f"{packed.dtype} [..., {packed.shape[-1]}] are not the bytes of [{rows}, {cols}] in {f}")
    lead, nt, kt, per = packed.shape[:-1], -(-rows // 16), -(-cols // 128), 128 // f.group
    p = packed.reshape(-1, nt, kt, 1024 + 32 * per)
    b = p[..., :1024].reshape(-1, nt, kt, 4, 16, 16)
    nibbles = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    g, nibble = _packed_places(f, packed.device)
    q = nibbles[:, :, :, g, :, nibble].permute(1, 2, 4, 3, 0)  # [matrix, row tile, row, column tile, column]
    if f.codes == B.MOE_PACKED_INT:
        v = q.float() - 8
    else:
        v = torch.tensor([*E2M1, *(-x for x in E2M1)], device=packed.device)[q.long()]
    s = p[..., 1024:].contiguous().view(B._TORCH_ACT[f.scale_dtype]).view(-1, nt, kt, 16, per).transpose(2, 3).float()
    v = v.reshape(*s.shape, f.group) * s[..., None]
    return v.reshape(-1, nt * 16, kt * 128)[:, :rows, :cols].reshape(*lead, rows, cols)


@dataclass
class PackedExperts:
    """The experts' weights in 4 bits: E packed matrices w_up [2 I, H] (gate rows
    first) and w_down [H, I]."""
    I: int
    format: B.PackedFormat
    w_up: torch.Tensor
    w_down: torch.Tensor


def pack_experts(w_up: torch.Tensor, w_down: torch.Tensor, f: B.PackedFormat) -> PackedExperts:
    """From weights [E, 2 I, H] and [E, H, I] in any float format."""
    return PackedExperts(I=w_down.shape[-1], format=f, w_up=pack_weights(w_up, f), w_down=pack_weights(w_down, f))


def run_layer_packed(b: Buffers, w: PackedExperts, h: torch.Tensor, stream=None) -> None:
    """Routing, the experts' products with 4-bit weights and the combine, from
    b.logits and the 16-bit rows b.x to b.out; h [T k, I] takes the inner rows."""
    route_assign_layout(b, stream)
    B.moe_expert_gemm_swiglu_packed(b.p, w.format, b.p.H, w.I, b.x, b.src, w.w_up, b.counts, b.expert_offsets, h,
                                    stream)
    B.moe_expert_gemm_packed(_act_out(b.p), w.format, w.I, b.p.H, h, None, w.w_down, b.counts, b.expert_offsets, b.y,
                             stream)
    combine(b, stream)


def layer_few_tokens_packed(b: Buffers, w: PackedExperts, ws: torch.Tensor, stream=None) -> None:
    """The same layer for a few tokens in two to four launches; `ws` has
    layer_packed_workspace(b, I) bytes."""
    B.moe_layer_few_tokens_packed(b.p, w.format, w.I, b.logits, b.x, w.w_up, w.w_down, b.idx, b.w, b.out, ws, stream)


def layer_packed_workspace(b: Buffers, I: int) -> torch.Tensor:
    return torch.empty(B.moe_layer_packed_workspace_bytes(b.p, I), dtype=torch.uint8, device=b.idx.device)


@dataclass
class WeightGrad:
    """The gradient of one of the experts' weights, dw [E, N, K] in fp32, and its
    workspace."""
    p: B.Problem
    N: int
    K: int
    dw: torch.Tensor
    ws: torch.Tensor


def allocate_weight_grad(b: Buffers, N: int, K: int) -> WeightGrad:
    E = b.p.E
    p = B.make_problem(b.p.T, E, b.p.k, b.p.H, b.p.R, b.p.act_dtype, b.p.flags | B.MOE_FLAG_OUT_F32)
    dev = b.idx.device
    return WeightGrad(p=p, N=N, K=K, dw=torch.empty(E, N, K, dtype=torch.float32, device=dev),
                      ws=torch.empty(B.moe_expert_weight_grad_workspace_bytes(p, K, N), dtype=torch.uint8, device=dev))


def expert_weight_grad(b: Buffers, g: WeightGrad, a: torch.Tensor, src: torch.Tensor | None, dy: torch.Tensor,
                       add: bool = False, stream=None) -> None:
    """g.dw from the products' 16-bit inputs a (send rows, or with src = b.src the
    token rows) and the gradient dy of their outputs; on top of g.dw with add."""
    B.moe_expert_weight_grad(g.p, g.K, g.N, a, src, dy, b.counts, b.expert_offsets, add, g.dw, g.ws, stream)
