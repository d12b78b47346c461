"""The 8-bit integer entry points at the ends of their arguments' range, on the host (no GPU). Fake
(never dereferenced) device addresses, so only where no GPU is visible."""
import ctypes

import pytest
import torch

from mxfp4_mixture_experts_route_amd import _lib

no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0,
                            reason="host-only validation tests use fake device addresses")
FAKE = ctypes.c_void_p(0x1000)
ESHAPE = _lib.MOE_ESHAPE
BF16 = _lib.MOE_BF16
INT_MAX = (1 << 31) - 1


def stack(E=1, N=48, K=100, glu=0):
    return ctypes.byref(_lib.I8ExpertsC(0x1000, 0x2000, None, E, N, K, glu))


@pytest.mark.parametrize("E,N,K,glu,tiles,chunks", [
    (1, INT_MAX, 1, 0, 1 << 27, 1), (1, INT_MAX - 14, 64, 0, 1 << 27, 1),
    (1, INT_MAX - 15, 65, 0, (1 << 27) - 1, 2), (1, INT_MAX - 1, 65536, 1, 1 << 27, 1024),
    (1024, INT_MAX, 65536, 0, 1 << 27, 1024)])
def test_packed_bytes_of_the_largest_matrices(E, N, K, glu, tiles, chunks):
    assert _lib.lib().i8_packed_bytes(E, N, K, glu) == E * tiles * chunks * 1024


def test_packed_bytes_past_63_bits_is_refused():
    assert _lib.lib().i8_packed_bytes(INT_MAX, INT_MAX, 65536, 0) == -1
    assert _lib.lib().i8_packed_bytes(1 << 16, INT_MAX, 65536, 0) == -1
    assert _lib.lib().i8_packed_bytes((1 << 16) - 1, INT_MAX, 65536, 0) == ((1 << 16) - 1) << 47


@no_gpu
@pytest.mark.parametrize("N,glu", [(INT_MAX, 0), (INT_MAX - 14, 0), (INT_MAX - 15, 0), (1 << 25, 0),
                                   (INT_MAX - 1, 1)])
def test_products_refuse_matrices_of_2_gb_and_more(N, glu):
    L, w = _lib.lib(), stack(N=N, K=64, glu=glu)
    assert L.i8_gemm(FAKE, FAKE, 3, w, FAKE, BF16, INT_MAX, None) == ESHAPE
    for rows in (3, 300):
        assert L.i8_linear(FAKE, BF16, 64, rows, w, FAKE, FAKE, FAKE, BF16, INT_MAX, None) == ESHAPE
    assert L.i8_moe_gemm(FAKE, FAKE, FAKE, 8, w, FAKE, FAKE, 16, 64, 0, 1.702, 7.0, FAKE,
                         None) == ESHAPE


@no_gpu
def test_linear_refuses_a_product_too_large_for_a_launch_before_it_quantizes():
    """The grid of a product has fewer than 2^32 threads. i8_linear says so as i8_gemm does, before
    its quantizer is launched (which reports another status here: there is no device)."""
    L, w = _lib.lib(), stack(N=1, K=1)
    assert L.i8_gemm(FAKE, FAKE, INT_MAX, w, FAKE, BF16, 1, None) == ESHAPE
    assert L.i8_linear(FAKE, BF16, 1, INT_MAX, w, FAKE, FAKE, FAKE, BF16, 1, None) == ESHAPE
