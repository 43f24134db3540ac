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
