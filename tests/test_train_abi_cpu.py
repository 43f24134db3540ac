"""Host-side checks of the training calls, without a GPU: bad arguments come
back as status codes, and from the binding as exceptions, before anything is
enqueued."""
import ctypes

import pytest
import torch

from combine_router_topk_amd import binding as B

BASE = 1 << 20
lib = B._lib


def refused(status, code, text):
    assert status == code, (status, B.moe_last_error())
    assert text in B.moe_last_error(), B.moe_last_error()


# ---- AdamW ----------------------------------------------------------------------

def adamw(h=None, n=1, array=True, control=None, **kw):
    step = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1, w_dtype=B.MOE_F32, g_dtype=B.MOE_F32, state_bits=32)
    step.update(h or {})
    t = dict(w=BASE, master=None, g=BASE * 2, m=BASE * 3, v=BASE * 4, m_scale=None, v_scale=None, n=16, weight_decay=0.1)
    if step["state_bits"] == 8:
        t.update(m_scale=BASE * 5, v_scale=BASE * 6)
    t.update(kw)
    a = (B._AdamWTensor * 1)(B._AdamWTensor(**t))
    return lib.moe_adamw_step(ctypes.byref(B.AdamW(**step)), a if array else None, n, control, None)


@pytest.mark.parametrize("h,text", [
    (dict(lr=float("nan")), "lr"), (dict(lr=float("inf")), "lr"), (dict(beta1=1.0), "beta1"), (dict(beta1=-0.1), "beta1"),
    (dict(beta2=1.5), "beta2"), (dict(beta2=float("nan")), "beta2"), (dict(eps=-1e-8), "eps"), (dict(eps=float("inf")), "eps"),
    (dict(step=0), "step=0"), (dict(w_dtype=0), "type 0"), (dict(g_dtype=4), "type 4"), (dict(state_bits=16), "state_bits=16")])
def test_adamw_refuses_bad_numbers(h, text):
    refused(adamw(h), B.MOE_ERR_INVALID_ARG, text)


@pytest.mark.parametrize("kw,text", [
    (dict(w=None), "w is NULL"), (dict(w=BASE + 8), "w is not 16-byte"), (dict(g=None), "g is NULL"),
    (dict(g=BASE + 4), "g is not 16-byte"), (dict(m=None), "m is NULL"), (dict(v=BASE + 8), "v is not 16-byte"),
    (dict(n=-1), "n=-1"), (dict(weight_decay=float("inf")), "weight_decay"), (dict(master=BASE), "a master beside"),
    (dict(m_scale=BASE), "scales beside"), (dict(v_scale=BASE), "scales beside")])
def test_adamw_refuses_bad_tensors(kw, text):
    refused(adamw(**kw), B.MOE_ERR_INVALID_ARG, text)


@pytest.mark.parametrize("kw,text", [
    (dict(m=BASE + 4), "m is not 8-byte"), (dict(v=BASE + 4), "v is not 8-byte"), (dict(m_scale=None), "m_scale is NULL"),
    (dict(v_scale=None), "v_scale is NULL"), (dict(v_scale=BASE + 2), "v_scale is not 4-byte")])
def test_adamw_refuses_bad_states_in_8_bits(kw, text):
    refused(adamw(dict(state_bits=8), **kw), B.MOE_ERR_INVALID_ARG, text)


def test_adamw_limits():
    refused(adamw(dict(w_dtype=B.MOE_F16, g_dtype=B.MOE_BF16)), B.MOE_ERR_UNSUPPORTED, "two different")
    refused(adamw(dict(w_dtype=B.MOE_F16), master=BASE + 8), B.MOE_ERR_INVALID_ARG, "master is not 16-byte")
    refused(adamw(n=-1), B.MOE_ERR_INVALID_ARG, "n=-1")
    refused(adamw(array=False), B.MOE_ERR_INVALID_ARG, "tensors is NULL")
    refused(adamw(control=ctypes.c_void_p(BASE + 2)), B.MOE_ERR_INVALID_ARG, "control is not 4-byte")
    refused(lib.moe_adamw_step(None, None, 0, None, None), B.MOE_ERR_INVALID_ARG, "h is NULL")
    t = (B._AdamWTensor * 1)(B._AdamWTensor(w=BASE, g=BASE, m=BASE, v=BASE, n=1 << 37))
    h = B.AdamW(1e-3, 0.9, 0.99, 1e-8, 1, B.MOE_F32, B.MOE_F32, 32)
    refused(lib.moe_adamw_step(ctypes.byref(h), t, 1, None, None), B.MOE_ERR_UNSUPPORTED, "is over")
    # nothing to do, whatever the pointers
    t[0] = B._AdamWTensor(n=0)
    assert lib.moe_adamw_step(ctypes.byref(h), t, 1, None, None) == B.MOE_OK
    assert lib.moe_adamw_step(ctypes.byref(h), None, 0, None, None) == B.MOE_OK


def test_adamw_tensors_are_checked_by_the_binding():
    one = lambda **kw: [dict(dict(w=torch.zeros(4), g=torch.zeros(4), m=torch.zeros(4), v=torch.zeros(4)), **kw)]  # noqa: E731
    with pytest.raises(ValueError, match="device tensor"):
        B.AdamWTensors(one())
    with pytest.raises(ValueError, match="dtype"):
        B.AdamWTensors(one(w=torch.zeros(4, dtype=torch.float64)))
    with pytest.raises(KeyError):
        B.AdamWTensors([dict(w=torch.zeros(4), g=torch.zeros(4))])
    B.moe_adamw_step(B.make_adamw(1e-3), B.AdamWTensors([]))  # no tensors: nothing happens


# ---- the weights' gradient --------------------------------------------------------

FAKE, OFF8 = ctypes.c_void_p(BASE), ctypes.c_void_p(BASE + 8)


def prob(**kw):
    d = dict(T=32, E=8, k=2, H=128, R=1, act_dtype=B.MOE_BF16, flags=0)
    d.update(kw)
    return ctypes.byref(B.make_problem(d["T"], d["E"], d["k"], d["H"], d["R"], d["act_dtype"], d["flags"]))


def grad(p=None, K=128, N=128, a=FAKE, src=None, dy=FAKE, counts=FAKE, off=FAKE, add=0, dw=FAKE, ws=None, n=0):
    return lib.moe_expert_weight_grad(p or prob(), K, N, a, src, dy, counts, off, add, dw, ws, n, None)


@pytest.mark.parametrize("kw,text", [
    (dict(K=0), "K=0"), (dict(K=12), "K=12"), (dict(N=0), "N=0"), (dict(N=-8), "N=-8"), (dict(N=20), "N=20"),
    (dict(a=None), "a is NULL"), (dict(a=OFF8), "a is not 16-byte"), (dict(dy=None), "dy is NULL"),
    (dict(dy=OFF8), "dy is not 16-byte"), (dict(dw=None), "dw is NULL"), (dict(dw=OFF8), "dw is not 16-byte"),
    (dict(counts=None), "counts is NULL"), (dict(off=None), "expert_offsets is NULL"),
    (dict(src=ctypes.c_void_p(BASE + 1)), "src is not 4-byte")])
def test_weight_grad_refusals(kw, text):
    refused(grad(**kw), B.MOE_ERR_INVALID_ARG, text)


def test_weight_grad_limits():
    refused(grad(add=1), B.MOE_ERR_UNSUPPORTED, "fp32 only")
    refused(grad(prob(E=1024), K=16392, N=16384), B.MOE_ERR_UNSUPPORTED, "too many tiles")
    n = ctypes.c_size_t(7)
    size = lambda p, K=128, N=128: lib.moe_expert_weight_grad_workspace_bytes(p, K, N, ctypes.byref(n))  # noqa: E731
    assert size(prob(E=64, T=16384), 4096, 4096) == B.MOE_OK and n.value == 0
    few = prob(T=16384, E=2)
    assert size(few) == B.MOE_OK and n.value > 2 * 2 * 128 * 128 * 4 and n.value < 300 << 20
    refused(grad(few), B.MOE_ERR_INVALID_ARG, "ws is NULL")
    refused(grad(few, ws=FAKE, n=n.value - 1), B.MOE_ERR_WORKSPACE, "workspace")
    refused(grad(few, ws=OFF8, n=n.value), B.MOE_ERR_INVALID_ARG, "ws is not 256-byte")
    refused(lib.moe_expert_weight_grad_workspace_bytes(prob(), 128, 128, None), B.MOE_ERR_INVALID_ARG, "bytes is NULL")
    refused(size(prob(), 12), B.MOE_ERR_INVALID_ARG, "K=12")
