"""NaN blocks of activation rows: they reach the outputs of their own row alone, and rows past the call's
M, whose scale bytes lie in the same padded layout, reach none."""
import pytest
import torch

from gpu_util import requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]


@pytest.fixture(scope="module")
def lib():
    import bit_w4a4_quantized_svdq_b200 as P
    return P


def _randn(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=g).to(torch.bfloat16)


@pytest.mark.parametrize("m,n,k", [(2, 136, 384), (20, 264, 4096), (100, 264, 4352), (130, 520, 640), (700, 384, 1152)])
def test_nan_activations_stay_in_their_rows(lib, m, n, k):
    x, w = _randn(m, m + 90, k), lib.svdq_quantize_mxfp4(_randn(n, n, k))
    clean = lib.svdq_quantize_mxfp4(x[:m])
    want = lib.svdq_linear_mxfp4(clean["codes"], clean["sf"], w["codes"], w["sf"])
    assert not bool(torch.isnan(want).any())
    x[m // 2, k - 1] = float("nan")
    x[m:, 5] = float("inf")                                   # rows behind the call's: NaN scales in the layout
    q = lib.svdq_quantize_mxfp4(x)
    wide = torch.full((m + 2, n), 5.0, dtype=torch.bfloat16, device="cuda")
    y = lib.svdq_linear_mxfp4(q["codes"][:m], q["sf"], w["codes"], w["sf"], out=wide[:m])
    rest = torch.arange(m, device="cuda") != m // 2
    assert bool(torch.isnan(y[m // 2]).all()) and torch.equal(y[rest], want[rest])
    assert bool((wide[m:] == 5.0).all())
    # the same for rows of the weight: n columns of a longer one
    w2 = _randn(n, n, k)
    longer = torch.cat([w2, torch.full((64, k), float("nan"), dtype=torch.bfloat16, device="cuda")])
    ql = lib.svdq_quantize_mxfp4(longer)
    assert torch.equal(lib.svdq_linear_mxfp4(clean["codes"], clean["sf"], ql["codes"][:n], ql["sf"]), want)
    back = lib.svdq_dequantize_mxfp4(q["codes"][:m], q["sf"])
    assert torch.equal(torch.isnan(back).any(1), ~rest)
