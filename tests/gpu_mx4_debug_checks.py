"""The debug library's store checks of the MXFP4 operators and the norms, made to fire
without any store leaving its buffer (the scheme of gpu_debug_checks.py).  The file name
keeps it out of the default collection; test_gpu_mx4_debug.py names it in a child process
that loads the debug library."""
import os

import pytest
import torch

from gpu_debug_checks import _armed, _check_prefix, _filled
from gpu_util import requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda,
              pytest.mark.skipif(os.environ.get("SVDQ_DEBUG", "0") in ("", "0"),
                                 reason="debug-library checks: run with SVDQ_DEBUG=1")]

MX_CODES, MX_SF, NORM_H, MX_VALUES, LINEAR = 15, 16, 32, 33, 34


@pytest.fixture(scope="module")
def P():
    import bit_w4a4_quantized_svdq_b200 as P
    assert P.load().svdq_debug_build() == 1, "the debug library must be the one loaded"
    return P


def _x(m, k, seed=1):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(m, k, device="cuda", generator=g).to(torch.bfloat16)


def test_quantiser_sites(P):
    m, k = 300, 384
    x = _x(m, k)
    want = P.svdq_quantize_mxfp4(x)
    for key, site, limit in (("codes", MX_CODES, (m // 2) * (k // 2)), ("sf", MX_SF, want["sf"].numel() // 2)):
        out = {n: _filled(torch.empty_like(t)) for n, t in want.items()}
        _armed(P, site, limit, lambda: P.svdq_quantize_mxfp4(x, out=out))
        _check_prefix(out[key], want[key], limit)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_dequantiser_site(P, fmt):
    m, k = 300, 384
    q = getattr(P, "svdq_quantize_" + fmt)(_x(m, k))
    back = getattr(P, "svdq_dequantize_" + fmt)
    want = back(q["codes"], q["sf"])
    y = _filled(torch.empty_like(want))
    _armed(P, MX_VALUES, (m // 2) * k, lambda: back(q["codes"], q["sf"], out=y))
    _check_prefix(y, want, (m // 2) * k * 2)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("k", [256, 640, 10240])              # several rows a CTA, one, two pieces a lane
def test_norm_sites(P, fmt, k):
    m = 300
    x, r, w = _x(m, k), _x(m, k, 2), torch.ones(k, device="cuda")
    norm = getattr(P, "svdq_rmsnorm_" + fmt)
    want = norm(x, w, r)
    row = want["codes"].shape[1]
    for key, site, limit, width in (("codes", MX_CODES, (m // 2) * row, 1), ("sf", MX_SF, want["sf"].numel() // 2, 1),
                                    ("h", NORM_H, (m // 2) * k, 2)):
        out = {n: _filled(torch.empty_like(t)) for n, t in want.items()}
        _armed(P, site, limit, lambda: norm(x, w, r, out=out))
        _check_prefix(out[key], want[key], limit * width)


@pytest.mark.parametrize("m,k", [(5, 1024), (60, 1024), (100, 8192)])   # the kernel whose M operand is the weight
def test_linear_few_rows_site(P, m, k):
    n = 392
    qa, qw = P.svdq_quantize_mxfp4(_x(m, k)), P.svdq_quantize_mxfp4(_x(n, k, 2))
    want = P.svdq_linear_mxfp4(qa["codes"], qa["sf"], qw["codes"], qw["sf"])
    y = _filled(torch.empty_like(want))
    limit = (m // 2) * n
    _armed(P, LINEAR, limit, lambda: P.svdq_linear_mxfp4(qa["codes"], qa["sf"], qw["codes"], qw["sf"], out=y))
    _check_prefix(y, want, limit * 2)


# 128-column tiles (100 rows of a short K among them) and 256-column tiles
@pytest.mark.parametrize("m,n,k", [(100, 384, 1024), (300, 384, 384), (4000, 5120, 384)])
def test_linear_many_rows_site(P, m, n, k):
    qa, qw = P.svdq_quantize_mxfp4(_x(m, k)), P.svdq_quantize_mxfp4(_x(n, k, 2))
    want = P.svdq_linear_mxfp4(qa["codes"], qa["sf"], qw["codes"], qw["sf"])
    y = _filled(torch.empty_like(want))
    # Y's TMA boxes: columns from n / 2 on are not stored
    _armed(P, LINEAR, n // 2, lambda: P.svdq_linear_mxfp4(qa["codes"], qa["sf"], qw["codes"], qw["sf"], out=y))
    assert torch.equal(y[:, :n // 2], want[:, :n // 2]) and bool((y[:, n // 2:].view(torch.int16) == -1).all())
