"""AdamW's numbers and sizes at the ends of what the kernel's fp32 and its grid hold,
without a GPU."""
import ctypes

import pytest

from combine_router_topk_amd import binding as B

lib = B._lib
BASE = 1 << 20


def step(n=16, w=None, **kw):
    """The status of a step with one tensor whose w is NULL unless given: numbers are
    looked at first."""
    h = dict(dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1, w_dtype=B.MOE_F32, g_dtype=B.MOE_F32, state_bits=32), **kw)
    t = (B._AdamWTensor * 1)(B._AdamWTensor(w=w, g=BASE, m=BASE, v=BASE, n=n, weight_decay=0.0))
    return lib.moe_adamw_step(ctypes.byref(B.AdamW(**h)), t, 1, None, None)


# the kernel takes them as fp32 numbers: 1e39 would be an infinity there, and every
# weight NaN; an eps of 1e-50 would be 0
@pytest.mark.parametrize("kw,text", [(dict(lr=1e39), "lr="), (dict(lr=-1e300), "lr="), (dict(lr=3.5e38), "lr="),
                                     (dict(eps=1e39), "eps="), (dict(eps=1e-50), "eps="), (dict(eps=5e-324), "eps=")])
def test_numbers_beyond_fp32_are_refused(kw, text):
    assert step(**kw) == B.MOE_ERR_INVALID_ARG and text in B.moe_last_error(), B.moe_last_error()


@pytest.mark.parametrize("kw", [dict(lr=3.4e38), dict(lr=1e-60), dict(lr=0.0), dict(lr=-0.1), dict(eps=0.0), dict(eps=1e-45),
                                dict(eps=3.4e38), dict(beta1=0.0, beta2=0.0), dict(beta1=1 - 2.0 ** -53)])
def test_numbers_within_it_are_taken(kw):
    assert step(**kw) == B.MOE_ERR_INVALID_ARG and "w is NULL" in B.moe_last_error(), B.moe_last_error()


def test_elements_of_a_tensor():
    most = 2 ** 35 - 2048
    assert step(n=most) == B.MOE_ERR_INVALID_ARG and "w is NULL" in B.moe_last_error()
    for n in (most + 1, 2 ** 35 - 1, 2 ** 35, 2 ** 63 - 1):
        assert step(n=n, w=BASE) == B.MOE_ERR_UNSUPPORTED and "is over" in B.moe_last_error(), n
