"""Sizes at the end of 32 bits in the calls that take experts' weights, without a
GPU: what the header calls too large comes back as MOE_ERR_UNSUPPORTED."""
import ctypes

import pytest

from combine_router_topk_amd import binding as B

lib = B._lib
FAKE = ctypes.c_void_p(1 << 20)
LARGEST = 2 ** 31 - 8  # the largest multiple of 8 in 32 bits


def prob(T=32, E=8, k=2, flags=0):
    return ctypes.byref(B.make_problem(T, E, k, 128, 1, B.MOE_BF16, flags))


# One side near 2^31: the other one's tiles decide, of which E * ceil(N / 128) *
# ceil(K / 256) has to stay below 2^23.
@pytest.mark.parametrize("T", [32, 1024, 16384])
@pytest.mark.parametrize("E,K,N", [(8, LARGEST, 8), (8, 8, LARGEST), (1, LARGEST, 8), (1, 8, LARGEST),
                                   (1, 2 ** 31 - 248, 8), (1, 8, 2 ** 31 - 120), (1024, LARGEST, LARGEST),
                                   (1, 8, 2 ** 30), (8, 8, 2 ** 27)])
def test_weight_grad_of_too_many_tiles(T, E, K, N):
    n = ctypes.c_size_t(7)
    assert lib.moe_expert_weight_grad_workspace_bytes(prob(T, E, 1), K, N, ctypes.byref(n)) == B.MOE_ERR_UNSUPPORTED
    assert "too many tiles" in B.moe_last_error() and n.value == 7
    assert lib.moe_expert_weight_grad(prob(T, E, 1), K, N, FAKE, None, FAKE, FAKE, FAKE, 0, FAKE, FAKE, 1 << 40,
                                      None) == B.MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("E,K,N", [(1, 2 ** 31 - 256, 8), (1, 8, 2 ** 30 - 128), (1, 2 ** 31 - 264, 128), (8, 8, 2 ** 27 - 128)])
def test_weight_grad_of_the_most_tiles(E, K, N):
    n = ctypes.c_size_t(7)
    tiles = -(-N // 128) * -(-K // 256)
    assert E * tiles < 2 ** 23 <= E * (tiles + 1)
    assert lib.moe_expert_weight_grad_workspace_bytes(prob(16384, E, 1), K, N, ctypes.byref(n)) == B.MOE_OK and n.value == 0


def test_products_with_packed_weights_of_too_many_rows_or_columns():
    f = ctypes.byref(B.make_packed_format(B.MOE_PACKED_INT, 64, B.MOE_F16))
    for K, N in ((LARGEST, 8), (8, LARGEST), (LARGEST, LARGEST)):
        assert lib.moe_expert_gemm_packed(prob(), f, K, N, FAKE, None, FAKE, FAKE, FAKE, FAKE, None) == B.MOE_ERR_UNSUPPORTED
    for K, I in ((LARGEST, 16), (8, 2 ** 31 - 16), (8, 2 ** 30)):
        assert lib.moe_expert_gemm_swiglu_packed(prob(), f, K, I, FAKE, None, FAKE, FAKE, FAKE, FAKE,
                                                 None) == B.MOE_ERR_UNSUPPORTED
    n = ctypes.c_size_t(7)
    for rows, cols in ((2 ** 31 - 1, 1), (1, 2 ** 31 - 1)):
        assert lib.moe_packed_weight_bytes(f, 1, rows, cols, ctypes.byref(n)) == B.MOE_ERR_UNSUPPORTED and n.value == 7
    wide = ctypes.byref(B.make_problem(4, 8, 2, 2 ** 31 - 16, 1, B.MOE_BF16))
    assert lib.moe_layer_packed_workspace_bytes(wide, 16, ctypes.byref(n)) == B.MOE_ERR_UNSUPPORTED
    assert lib.moe_layer_packed_workspace_bytes(prob(), 2 ** 31 - 16, ctypes.byref(n)) == B.MOE_ERR_UNSUPPORTED
