"""Host-side checks of the calls with packed weights, without a GPU."""
import ctypes

import pytest
import torch

from combine_router_topk_amd import binding as B

FAKE, OFF8 = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 8)
lib = B._lib


def prob(**kw):
    d = dict(T=32, E=8, k=2, H=128, R=1, act_dtype=B.MOE_BF16, flags=0)
    d.update(kw)
    return ctypes.byref(B.make_problem(d["T"], d["E"], d["k"], d["H"], d["R"], d["act_dtype"], d["flags"]))


def fmt(codes=B.MOE_PACKED_INT, group=64, scale_dtype=B.MOE_F16):
    return ctypes.byref(B.make_packed_format(codes, group, scale_dtype))


def refused(status, code, text):
    assert status == code, (status, B.moe_last_error())
    assert text in B.moe_last_error(), B.moe_last_error()


def gemm(p=None, f=None, K=128, N=128, a=FAKE, src=None, w=FAKE, counts=FAKE, off=FAKE, y=FAKE):
    return lib.moe_expert_gemm_packed(p or prob(), f or fmt(), K, N, a, src, w, counts, off, y, None)


def swiglu(p=None, f=None, K=128, I=128, a=FAKE, src=None, w=FAKE, counts=FAKE, off=FAKE, h=FAKE):
    return lib.moe_expert_gemm_swiglu_packed(p or prob(), f or fmt(), K, I, a, src, w, counts, off, h, None)


def layer(p=None, f=None, I=64, logits=FAKE, x=FAKE, wu=FAKE, wd=FAKE, idx=FAKE, w=FAKE, out=FAKE, ws=FAKE, n=1 << 30):
    return lib.moe_layer_few_tokens_packed(p or prob(), f or fmt(), I, logits, x, wu, wd, idx, w, out, ws, n, None)


@pytest.mark.parametrize("call", [gemm, swiglu, layer])
@pytest.mark.parametrize("kw,text", [(dict(codes=0), "codes=0"), (dict(codes=3), "codes=3"), (dict(group=16), "group=16"),
                                     (dict(group=0), "group=0"), (dict(group=256), "group=256"),
                                     (dict(scale_dtype=3), "scale_dtype=3")])
def test_format_refusals(call, kw, text):
    refused(call(f=fmt(**kw)), B.MOE_ERR_INVALID_ARG, text)


@pytest.mark.parametrize("call", [gemm, swiglu])
@pytest.mark.parametrize("kw,text", [
    (dict(K=0), "K=0"), (dict(K=12), "K=12"), (dict(K=-8), "K=-8"), (dict(a=None), "a is NULL"),
    (dict(a=OFF8), "a is not 16-byte"), (dict(w=None), "w is NULL"), (dict(w=OFF8), "w is not 16-byte"),
    (dict(counts=None), "counts is NULL"), (dict(off=None), "expert_offsets is NULL"),
    (dict(src=ctypes.c_void_p(1 << 20 | 1)), "src is not 4-byte")])
def test_product_refusals(call, kw, text):
    refused(call(**kw), B.MOE_ERR_INVALID_ARG, text)


def test_product_sizes():
    for N in (0, 12, -8):
        refused(gemm(N=N), B.MOE_ERR_INVALID_ARG, f"N={N}")
    for I in (0, 8, -16):
        refused(swiglu(I=I), B.MOE_ERR_INVALID_ARG, f"I={I}")
    refused(gemm(y=None), B.MOE_ERR_INVALID_ARG, "y is NULL")
    refused(swiglu(h=OFF8), B.MOE_ERR_INVALID_ARG, "h is not 16-byte")
    refused(gemm(K=(1 << 24) + 8), B.MOE_ERR_UNSUPPORTED, "K=")
    refused(gemm(N=(1 << 24) + 8), B.MOE_ERR_UNSUPPORTED, "tiles")
    refused(swiglu(I=(1 << 23) + 16), B.MOE_ERR_UNSUPPORTED, "tiles")
    refused(gemm(prob(T=(1 << 24) - 1, k=1), N=1 << 24), B.MOE_ERR_UNSUPPORTED, "tiles")
    refused(lib.moe_expert_gemm_packed(prob(), None, 128, 128, *(FAKE,) * 3, FAKE, FAKE, FAKE, None),
            B.MOE_ERR_INVALID_ARG, "format is NULL")
    # no rows: nothing to do, whatever the pointers
    assert gemm(prob(T=0), a=None, w=None, counts=None, off=None, y=None) == B.MOE_OK
    assert swiglu(prob(T=0), a=None, w=None, counts=None, off=None, h=None) == B.MOE_OK


@pytest.mark.parametrize("name", ["logits", "x", "wu", "wd", "idx", "w", "out", "ws"])
def test_layer_refusals(name):
    refused(layer(**{name: None}), B.MOE_ERR_INVALID_ARG, "is NULL")
    refused(layer(n=16), B.MOE_ERR_WORKSPACE, "workspace")
    refused(layer(prob(H=24)), B.MOE_ERR_INVALID_ARG, "H=24")
    refused(layer(I=24), B.MOE_ERR_INVALID_ARG, "I=24")
    refused(layer(prob(T=65)), B.MOE_ERR_UNSUPPORTED, "T=65")
    refused(layer(ws=OFF8), B.MOE_ERR_INVALID_ARG, "ws is not 256-byte")
    assert layer(prob(T=0), logits=None, x=None, wu=None, wd=None, idx=None, w=None, out=None, ws=None, n=0) == B.MOE_OK


def test_bytes():
    n = ctypes.c_size_t(7)
    call = lambda f, E=2, r=17, c=129: lib.moe_packed_weight_bytes(f, E, r, c, ctypes.byref(n))  # noqa: E731
    for group, tile in ((128, 1056), (64, 1088), (32, 1152)):
        assert call(fmt(group=group)) == B.MOE_OK and n.value == 2 * 2 * 2 * tile
    for kw in (dict(E=0), dict(r=0), dict(c=0)):
        refused(call(fmt(), **kw), B.MOE_ERR_INVALID_ARG, "at least 1")
    for kw in (dict(E=1025), dict(r=(1 << 24) + 1), dict(c=(1 << 24) + 1)):
        refused(call(fmt(), **kw), B.MOE_ERR_UNSUPPORTED, "over")
    refused(lib.moe_packed_weight_bytes(fmt(), 1, 1, 1, None), B.MOE_ERR_INVALID_ARG, "bytes is NULL")
    refused(lib.moe_layer_packed_workspace_bytes(prob(), 64, None), B.MOE_ERR_INVALID_ARG, "bytes is NULL")
    assert call(fmt(), E=1024, r=1 << 24, c=1 << 24) == B.MOE_OK and n.value == 1024 * (1 << 20) * (1 << 17) * 1088


def test_binding_checks_sizes():
    p, f = B.make_problem(4, 2, 1, 32, 1, B.MOE_F16), B.make_packed_format(B.MOE_PACKED_E2M1, 32, B.MOE_F16)
    with pytest.raises(ValueError, match="device tensor"):
        B.moe_expert_gemm_packed(p, f, 32, 16, torch.zeros(4, 32, dtype=torch.float16), None, None, None, None, None)
