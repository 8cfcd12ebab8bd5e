"""SwiGLU with sums in fp32 at any size is a choice of the fp8 products with block scales: they check its arguments as
SwiGLU's, and every other grouped product refuses it (placeholder pointers that are never dereferenced; no GPU is needed)."""
import ctypes

import pytest
import torch

import w4a16_routed_expert_moe_amd as moe
from w4a16_routed_expert_moe_amd import _lib

OK, NULL, SHAPE, UNSUP, ALIGN = 0, 1, 2, 3, 4
P = ctypes.c_void_p
A, ODD = P(0x10000), P(0x10002)

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder-pointer checks run without a GPU")


def _desc():
    return ctypes.byref(moe.MoeLayerDesc.make(4096, 2048, 256, 6, 1))


@pytest.mark.parametrize("N,act,out,status", [(4096, 3, None, NULL), (4096, 3, ODD, ALIGN), (192, 3, A, SHAPE), (4096, 2, A, UNSUP), (4096, 4, A, UNSUP),
                                              (4096, -1, A, UNSUP)])
def test_arguments(N, act, out, status):
    assert moe.MOE_ACT_SWIGLU_F32 == 3
    assert _lib.lib().moe_fp8s_grouped_gemm(_desc(), 4, A, A, A, 4, N, 4096, A, A, A, act, out, None) == status


def test_without_tokens():
    assert _lib.lib().moe_fp8s_grouped_gemm(_desc(), 0, None, None, None, 0, 4096, 4096, None, None, None, 3, None, None) == OK


def test_other_products_refuse_it():
    L = _lib.lib()
    assert L.moe_bf16_grouped_gemm(_desc(), 4, A, A, 4, 4096, 4096, A, A, 3, A, A, None) == UNSUP
    assert L.moe_w8a8_grouped_gemm(_desc(), 4, A, A, A, 4, 4096, 4096, A, A, A, 3, A, None) == UNSUP
    assert L.moe_w4a16_grouped_gemm(_desc(), 4, A, A, 4, None, 4096, 4096, A, A, A, 3, A, None) == UNSUP
    assert L.moe_mxfp4_grouped_gemm(_desc(), 4, A, A, 4, 4096, 4096, A, A, A, 3, A, None) == UNSUP
    assert L.moe_w4a8_grouped_gemm(_desc(), 4, A, A, A, 4, 4096, 4096, A, A, A, 3, A, None) == UNSUP
