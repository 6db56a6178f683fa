"""The largest sizes and arguments of the MXFP4 calls and the norms, at the C entries, on CPU (no launch:
the pointers are made up, and without a device a call that passes its checks answers so)."""
import pytest
import torch

from bit_w4a4_quantized_svdq_b200 import _lib

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers: CPU only")

P = 0x10000
OK = (_lib.SVDQ_ERR_NO_DEVICE,)


def _mx(name, m, k, ld):
    lib = _lib.load()
    if "dequantize" in name:
        return getattr(lib, name)(P, P, m, k, P, ld, None)
    return getattr(lib, name)(P, m, k, ld, P, P, None)


@pytest.mark.parametrize("name", ["svdq_quantize_mxfp4", "svdq_dequantize_mxfp4", "svdq_dequantize_mxfp8"])
@pytest.mark.parametrize("m,k", [(1 << 40, 1 << 30), ((1 << 40) - 127, 1 << 30), (1 << 40, 1 << 29), (1 << 31, 128),
                                 (128, 1 << 31), (1 << 22, 1 << 20)])
def test_sizes_past_the_unit_count_are_refused(name, m, k):
    """Among them the product that wraps around 64 bits."""
    assert _mx(name, m, k, k) == _lib.SVDQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("name", ["svdq_quantize_mxfp4", "svdq_dequantize_mxfp4", "svdq_dequantize_mxfp8"])
@pytest.mark.parametrize("m,k", [(1, 128), (128, 1 << 30), (0x7FFF0000, 128), (110000, 20480)])
def test_sizes_within_it_are_taken(name, m, k):
    assert _mx(name, m, k, k) in OK


@pytest.mark.parametrize("name", ["svdq_rmsnorm_mxfp8", "svdq_rmsnorm_mxfp4"])
def test_norm_takes_any_positive_finite_eps(name):
    def call(eps):
        return getattr(_lib.load(), name)(P, 4, 256, 256, None, 0, P, 1, eps, None, 0, P, P, None)

    for eps in (1e-45, 1e-38, 1e-6, 1.0, 3.2e38, 3.4028234e38):
        assert call(eps) in OK, eps
    for eps in (0.0, -0.0, -1e-6, float("inf"), float("-inf"), float("nan"), 1e-46):
        assert call(eps) == _lib.SVDQ_ERR_INVALID_ARG, eps
