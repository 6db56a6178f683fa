"""MXFP4 linear and norms at the edges of their launch plans, against the oracle in 64 bits."""
import numpy as np
import pytest
import torch

import synthetic as S
from oracle import svdq_oracle as O
from gpu_util import dev_bits, host_bits, requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]


@pytest.fixture(scope="module")
def lib():
    import bit_w4a4_quantized_svdq_b200 as P
    return P


# ------------------------------------------------------------------------------------------ linear
# Columns that end inside a warp's share (lanes without a store before a cluster barrier), K sliced
# over 2, 4 and 8 CTAs and whole; tiles whose second half of the columns is missing or partial.
@pytest.mark.parametrize("m,n,k", [(1, 8, 4096), (3, 24, 8192), (5, 120, 1024), (12, 136, 2048), (30, 200, 4096),
                                   (60, 264, 16640), (100, 328, 4352), (128, 8, 8192), (130, 8, 640), (257, 136, 384),
                                   (300, 200, 256), (4200, 9416, 256), (4200, 9352, 384)])
def test_linear_ragged_columns(lib, m, n, k):
    x_bits, w_bits = S.random_bf16((m, k), m + n, 1.0), S.random_bf16((n, k), n + k, 0.02)
    bias = S.random_bf16((n,), 7, 0.05)
    qa, qw = lib.svdq_quantize_mxfp4(dev_bits(x_bits)), lib.svdq_quantize_mxfp4(dev_bits(w_bits))
    wide = torch.full((m, n + 64), 5.0, dtype=torch.bfloat16, device="cuda")
    args = (qa["codes"], qa["sf"], qw["codes"], qw["sf"], dev_bits(bias))
    y = lib.svdq_linear_mxfp4(*args, out=wide[:, :n])
    rows = np.unique(np.concatenate([np.arange(min(m, 40)), np.random.default_rng(0).choice(m, min(m, 60), replace=False),
                                     [m - 1]]))
    a = O.mx4_dequantize(*O.mx_quantize_values(O.bf16_to_f64(x_bits[rows]), "mxfp4"))
    w = O.mx4_dequantize(*O.mx_quantize_values(O.bf16_to_f64(w_bits), "mxfp4"))
    b = O.bf16_to_f64(bias)[None, :]
    y64 = a @ w.T + b
    # one rounding to bf16 and K / 64 + 8 fp32 additions of exact products, each at most a unit of 2^-23
    bound = np.abs(y64) * 2.0 ** -8 * (1 + 2.0 ** -8) + (k / 64 + 8) * 2.0 ** -23 * (np.abs(a) @ np.abs(w).T + np.abs(b))
    err = np.abs(O.bf16_to_f64(host_bits(y[torch.from_numpy(rows).cuda()])) - y64)
    assert (err <= bound).all(), f"{(err > bound).sum()} of {err.size} outputs off"
    assert bool((wide[:, n:] == 5.0).all())
    for _ in range(5):
        assert torch.equal(lib.svdq_linear_mxfp4(*args), y)
    assert lib.svdq_device_error() == 0
