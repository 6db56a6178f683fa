"""The MXFP4 linear's launch plans that few shapes reach, every output against a 64-bit product of the
operands' values (read back from their codes, which test_gpu_mx4.py compares bit for bit):

* rows as the MMA's columns (8 to 128 of them), K sliced over 2 and 8 CTAs;
* 128-column tiles with several tiles a pair of CTAs (columns few, rows many);
* operands past one band of the tile walk, along the rows and along the columns."""
import pytest
import torch

from gpu_util import requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]


@pytest.fixture(scope="module")
def lib():
    import bit_w4a4_quantized_svdq_b200 as P
    return P


def _randn(m, k, seed, scale):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (scale * torch.randn(m, k, device="cuda", generator=g)).to(torch.bfloat16)


FEW_SLICED = [(8, 10008, 4352), (3, 1160, 16384), (15, 400, 16640), (13, 10008, 2048), (27, 136, 16512),
              (32, 10008, 1024), (64, 264, 16384), (33, 12000, 2048), (72, 10008, 4352), (120, 10008, 4352),
              (115, 264, 16384), (128, 1160, 20480)]
NARROW_TILES = [(40000, 128, 256), (40001, 72, 640), (60000, 64, 384), (58000, 8, 1408), (12544, 384, 1152),
                (12500, 320, 1280)]
BANDS = [(2816, 2560, 65536), (2560, 2816, 65536), (4096, 4104, 22528)]


@pytest.mark.parametrize("m,n,k", FEW_SLICED + NARROW_TILES + BANDS)
def test_linear_plan(lib, m, n, k):
    qa, qw = lib.svdq_quantize_mxfp4(_randn(m, k, m, 1.0)), lib.svdq_quantize_mxfp4(_randn(n, k, n + 1, 0.02))
    bias = _randn(1, n, 7, 0.05).view(-1)
    args = (qa["codes"], qa["sf"], qw["codes"], qw["sf"], bias)
    wide = torch.full((m + 1, n + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    y = lib.svdq_linear_mxfp4(*args, out=wide[:m, :n])
    w = lib.svdq_dequantize_mxfp4(qw["codes"], qw["sf"]).double().t()
    wa, b = w.abs(), bias.double()
    for r0 in range(0, m, 1024):
        a = lib.svdq_dequantize_mxfp4(qa["codes"], qa["sf"])[r0:r0 + 1024].double()
        y64 = a @ w + b
        # one rounding to bf16, and K / 64 + 8 fp32 additions of exact products, each at most a unit of 2^-23
        bound = y64.abs() * 2.0 ** -8 * (1 + 2.0 ** -8) + (k / 64 + 8) * 2.0 ** -23 * (a.abs() @ wa + b.abs())
        err = (y[r0:r0 + 1024].double() - y64).abs()
        bad = (~(err <= bound)).nonzero()
        assert bad.numel() == 0, f"{len(bad)} outputs off in rows {r0}.., first {bad[:4].tolist()}"
    assert bool((wide[m] == 5.0).all()) and bool((wide[:, n:] == 5.0).all())
    want = y.clone()
    for _ in range(10):
        assert torch.equal(lib.svdq_linear_mxfp4(*args), want)
    assert lib.svdq_device_error() == 0
