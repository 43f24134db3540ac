"""Host-side checks of the layer's entry points, without a GPU: bad arguments
come back as status codes, and from the binding as exceptions, before
anything is enqueued."""
import ctypes

import pytest
import torch

from combine_router_topk_amd import binding as B

FAKE = ctypes.c_void_p(1 << 20)
OFF8 = ctypes.c_void_p((1 << 20) + 8)
OFF4 = ctypes.c_void_p((1 << 20) + 4)
lib = B._lib


def prob(**kw):
    d = dict(T=32, E=8, k=2, H=128, R=1, act_dtype=B.MOE_BF16, flags=0)
    d.update(kw)
    return ctypes.byref(B.make_problem(d["T"], d["E"], d["k"], d["H"], d["R"], d["act_dtype"], d["flags"]))


def refused(status, code, text):
    assert status == code, (status, B.moe_last_error())
    assert text in B.moe_last_error(), B.moe_last_error()


def norm(p=None, x=FAKE, res=FAKE, gamma=FAKE, eps=1e-6, h=FAKE, y=OFF8, q=FAKE, qs=FAKE, rstd=FAKE):
    return lib.moe_rms_norm(p or prob(), x, res, gamma, eps, h, y, q, qs, rstd, None)


@pytest.mark.parametrize("kw,text", [
    (dict(x=None), "x is NULL"), (dict(gamma=None), "gamma is NULL"), (dict(h=None), "residual and h"),
    (dict(res=None), "residual and h"), (dict(q=None), "q and q_scale"), (dict(qs=None), "q and q_scale"),
    (dict(y=None, q=None, qs=None), "both NULL"), (dict(y=FAKE), "same buffer"), (dict(eps=-1.0), "eps"),
    (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps"), (dict(x=OFF8), "x is not 16-byte"),
    (dict(res=OFF8), "residual is not"), (dict(h=OFF8, y=FAKE), "h is not"), (dict(y=OFF8), "y is not 16-byte"),
    (dict(y=None, q=OFF4), "q is not 8-byte"), (dict(y=None, qs=ctypes.c_void_p(1 << 20 | 2)), "q_scale is not"),
    (dict(y=None, rstd=ctypes.c_void_p(1 << 20 | 1)), "rstd is not")])
def test_norm_refusals(kw, text):
    refused(norm(**kw), B.MOE_ERR_INVALID_ARG, text)


def test_norm_limits():
    refused(norm(prob(H=B.MOE_MAX_NORM_H + 8)), B.MOE_ERR_UNSUPPORTED, "is over")
    refused(norm(prob(H=12)), B.MOE_ERR_INVALID_ARG, "multiple of 8")
    n = ctypes.c_size_t(7)
    assert lib.moe_rms_norm_workspace_bytes(prob(H=B.MOE_MAX_NORM_H), ctypes.byref(n)) == B.MOE_OK and n.value > 0
    refused(lib.moe_rms_norm_workspace_bytes(prob(), None), B.MOE_ERR_INVALID_ARG, "bytes is NULL")
    refused(lib.moe_rms_norm_workspace_bytes(prob(H=B.MOE_MAX_NORM_H + 8), ctypes.byref(n)),
            B.MOE_ERR_UNSUPPORTED, "is over")
    assert lib.moe_rms_norm_workspace_bytes(prob(T=0), ctypes.byref(n)) == B.MOE_OK and n.value == 0
    # no rows: nothing to do, whatever the pointers
    assert norm(prob(T=0), *(None,) * 3, h=None, y=None, q=None, qs=None, rstd=None) == B.MOE_OK


@pytest.mark.parametrize("name", ["dy", "h", "gamma", "rstd", "dx", "dgamma", "ws"])
def test_norm_backward_refusals(name):
    a = dict(dy=FAKE, dh=None, h=FAKE, gamma=FAKE, rstd=FAKE, dx=FAKE, dgamma=FAKE, ws=FAKE)
    call = lambda p=None, n=1 << 30, **kw: lib.moe_rms_norm_backward(p or prob(), *{**a, **kw}.values(), n, None)  # noqa: E731
    refused(call(**{name: None}), B.MOE_ERR_INVALID_ARG, f"{name} is NULL")
    refused(call(dh=OFF8), B.MOE_ERR_INVALID_ARG, "dh is not 16-byte")
    refused(call(ws=OFF8), B.MOE_ERR_INVALID_ARG, "ws is not 256-byte")
    refused(call(n=16), B.MOE_ERR_WORKSPACE, "workspace")


def gemm(p=None, K=128, N=128, a=FAKE, sa=FAKE, src=None, w=FAKE, sw=FAKE, counts=FAKE, off=FAKE, y=FAKE):
    return lib.moe_expert_gemm(p or prob(), K, N, a, sa, src, w, sw, counts, off, y, None)


def swiglu(p=None, K=128, I=128, a=FAKE, sa=FAKE, src=None, w=FAKE, sw=FAKE, counts=FAKE, off=FAKE, q=FAKE,
           qs=FAKE):
    return lib.moe_expert_gemm_swiglu(p or prob(), K, I, a, sa, src, w, sw, counts, off, q, qs, None)


@pytest.mark.parametrize("call", [gemm, swiglu])
@pytest.mark.parametrize("kw,text", [
    (dict(K=0), "K=0"), (dict(K=24), "K=24"), (dict(K=-16), "K=-16"), (dict(a=None), "a is NULL"),
    (dict(a=OFF8), "a is not 16-byte"), (dict(sa=None), "a_scale is NULL"), (dict(w=None), "w is NULL"),
    (dict(w=OFF8), "w is not 16-byte"), (dict(sw=None), "w_scale is NULL"), (dict(counts=None), "counts is NULL"),
    (dict(off=None), "expert_offsets is NULL"), (dict(src=ctypes.c_void_p(1 << 20 | 1)), "src is not 4-byte")])
def test_product_refusals(call, kw, text):
    refused(call(**kw), B.MOE_ERR_INVALID_ARG, text)


def test_product_sizes():
    for N in (0, 12, -8):
        refused(gemm(N=N), B.MOE_ERR_INVALID_ARG, f"N={N}")
    for I in (0, 8, -16):
        refused(swiglu(I=I), B.MOE_ERR_INVALID_ARG, f"I={I}")
    refused(gemm(y=None), B.MOE_ERR_INVALID_ARG, "y is NULL")
    refused(gemm(y=OFF8), B.MOE_ERR_INVALID_ARG, "y is not")
    refused(swiglu(q=None), B.MOE_ERR_INVALID_ARG, "q is NULL")
    refused(swiglu(qs=None), B.MOE_ERR_INVALID_ARG, "q_scale is NULL")
    # beyond 32-bit offsets: an expert's codes, the gathered rows' codes, 2 I
    refused(gemm(K=1 << 16, N=1 << 16), B.MOE_ERR_UNSUPPORTED, "32-bit")
    refused(gemm(prob(T=1 << 20), K=4096, src=FAKE), B.MOE_ERR_UNSUPPORTED, "32-bit")
    refused(swiglu(I=(1 << 31) - 16), B.MOE_ERR_UNSUPPORTED, "32-bit")
    # no rows: nothing to do
    none = dict.fromkeys(("a", "sa", "w", "sw", "counts", "off"))
    assert gemm(prob(T=0), y=None, **none) == B.MOE_OK
    assert swiglu(prob(T=0), q=None, qs=None, **none) == B.MOE_OK


def layer(p=None, I=128, logits=FAKE, x=FAKE, wu=FAKE, su=FAKE, wd=FAKE, sd=FAKE, idx=FAKE, w=FAKE, out=FAKE,
          ws=FAKE, n=1 << 30):
    return lib.moe_layer_few_tokens(p or prob(), I, logits, x, wu, su, wd, sd, idx, w, out, ws, n, None)


@pytest.mark.parametrize("kw,text", [
    (dict(I=0), "I=0"), (dict(I=24), "I=24"), (dict(su=None), "s_up and s_down"), (dict(sd=None), "s_up and s_down"),
    (dict(logits=None), "logits is NULL"), (dict(x=None), "x is NULL"), (dict(x=OFF8), "x is not 16-byte"),
    (dict(wu=None), "w_up is NULL"), (dict(wu=OFF8), "w_up is not"), (dict(wd=None), "w_down is NULL"),
    (dict(wd=OFF8), "w_down is not"), (dict(idx=None), "idx is NULL"), (dict(w=None), "w is NULL"),
    (dict(out=None), "out is NULL"), (dict(out=OFF8), "out is not"), (dict(ws=None), "ws is NULL"),
    (dict(ws=OFF8), "ws is not 256-byte")])
def test_layer_refusals(kw, text):
    refused(layer(**kw), B.MOE_ERR_INVALID_ARG, text)


def test_layer_limits():
    refused(layer(prob(T=65)), B.MOE_ERR_UNSUPPORTED, "T=65")
    refused(layer(prob(H=136)), B.MOE_ERR_INVALID_ARG, "H=136")
    refused(layer(n=16), B.MOE_ERR_WORKSPACE, "workspace")
    assert layer(prob(T=0), 128, *(None,) * 10, n=0) == B.MOE_OK
    n = ctypes.c_size_t(0)
    assert lib.moe_layer_workspace_bytes(prob(), 128, ctypes.byref(n)) == B.MOE_OK
    assert n.value >= 32 * 2 * 128 * 2 and n.value % 256 == 0
    refused(lib.moe_layer_workspace_bytes(prob(), 128, None), B.MOE_ERR_INVALID_ARG, "bytes is NULL")
    refused(lib.moe_layer_workspace_bytes(prob(T=65), 128, ctypes.byref(n)), B.MOE_ERR_UNSUPPORTED, "T=65")


def test_layer_rows_past_the_kernels_counts():
    """Rows whose count of elements, T H, or whose columns 32 bits do not hold
    are refused: at T = 64, H = 2^26 + 16 the count came to 1024. Refused
    before the workspace is looked at, so nothing is enqueued."""
    most, n = 1 << 24, ctypes.c_size_t(0)
    one = dict(T=64, E=1, k=1)
    for H in (most + 16, (1 << 25) + 16, (1 << 26) + 16, (1 << 31) - 16):
        refused(layer(prob(H=H, **one), 16, n=0), B.MOE_ERR_UNSUPPORTED, f"H={H}")
        refused(lib.moe_layer_workspace_bytes(prob(H=H, **one), 16, ctypes.byref(n)), B.MOE_ERR_UNSUPPORTED, f"H={H}")
    for I in (most + 16, (1 << 31) - 16):
        refused(layer(prob(**one), I, n=0), B.MOE_ERR_UNSUPPORTED, f"I={I}")
    # the widest rows that are taken, with the shares' sums in the workspace
    # (shares from H I = 2^29 on, which I = 32 misses by 512)
    assert lib.moe_layer_workspace_bytes(prob(H=most - 16, **one), 48, ctypes.byref(n)) == B.MOE_OK
    assert n.value >= 4 * 64 * (most - 16) * 4
    assert lib.moe_layer_workspace_bytes(prob(H=most, **one), most, ctypes.byref(n)) == B.MOE_OK
    assert n.value >= 64 * most * 2


def test_binding_checks_tensors_before_the_library():
    p = B.make_problem(4, 8, 2, 64, 1, B.MOE_BF16)
    with pytest.raises(ValueError, match="device tensor"):
        B.moe_rms_norm(p, torch.zeros(4, 64, dtype=torch.bfloat16), None, None, 1e-6, None, None, None, None, None,
                       stream=0)
    with pytest.raises(B.MoeError, match="both NULL"):
        B.moe_rms_norm(p, None, None, None, 1e-6, None, None, None, None, None, stream=0)
    with pytest.raises(B.MoeError, match="a is NULL"):
        B.moe_expert_gemm(p, 64, 64, *(None,) * 8, stream=0)
    with pytest.raises(B.MoeError, match="a is NULL"):
        B.moe_expert_gemm_swiglu(p, 64, 64, *(None,) * 9, stream=0)
    with pytest.raises(B.MoeError, match="logits is NULL"):
        B.moe_layer_few_tokens(p, 64, *(None,) * 10, stream=0)
    with pytest.raises(B.MoeError, match="dgamma is NULL"):
        B.moe_rms_norm_backward(p, *(None,) * 8, stream=0)


def test_limits_match_the_header():
    import os
    import re
    from conftest import ROOT
    text = open(os.path.join(ROOT, "include", "moe_route.h")).read()
    for name in ("MOE_SCALE_BLOCK", "MOE_MAX_NORM_H", "MOE_MAX_FEW_TOKENS"):
        m = re.search(rf"{name} = (\d+)", text)
        assert m and int(m.group(1)) == getattr(B, name), name
    assert [B.scale_blocks(c) for c in (1, 128, 129)] == [1, 1, 2]


def test_flags_match_the_header():
    import os
    import re
    from conftest import ROOT
    text = open(os.path.join(ROOT, "include", "moe_route.h")).read()
    for name in ("MOE_FLAG_GREEDY_ID_ORDER", "MOE_FLAG_OUT_F32", "MOE_FLAG_EXACT_SUMS"):
        m = re.search(rf"{name} = 1u << (\d+)", text)
        assert m and 1 << int(m.group(1)) == getattr(B, name), name
    # every call takes the known flags, and no other
    known, n = B.MOE_FLAG_EXACT_SUMS | B.MOE_FLAG_OUT_F32, ctypes.c_size_t(0)
    assert gemm(prob(T=0, flags=known), y=None, **dict.fromkeys(("a", "sa", "w", "sw", "counts", "off"))) == B.MOE_OK
    assert layer(prob(T=0, flags=known), 128, *(None,) * 10, n=0) == B.MOE_OK
    assert lib.moe_workspace_bytes(prob(flags=known), ctypes.byref(n)) == B.MOE_OK
    refused(gemm(prob(flags=B.MOE_FLAG_EXACT_SUMS << 1)), B.MOE_ERR_INVALID_ARG, "unknown flag")
