"""The norms where a CTA walks several rows: the next row's loads in flight, the partial sums'
two buffers in turn, grids of several waves.

Every row is compared with the same row in a launch of 128 rows (one round a CTA, the shapes that
test_gpu_mx4.py holds to the oracle), sampled rows with the oracle in 64 bits, and the whole of h
with the sum rounded once."""
import numpy as np
import pytest
import torch

import synthetic as S
from oracle import svdq_oracle as O
from gpu_util import check_sf, host_bits, requires_cuda
from test_gpu_mx4 import _check_norm, _natural_scales

pytestmark = [pytest.mark.gpu, requires_cuda]


@pytest.fixture(scope="module")
def lib():
    import bit_w4a4_quantized_svdq_b200 as P
    return P


def _randn(m, k, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(m, k, device="cuda", generator=g)
    # no two rows alike in size, so that another row's sum shows in every code
    return (scale * x * torch.exp2(torch.randint(-3, 4, (m, 1), device="cuda", generator=g).float())).to(torch.bfloat16)


def _sampled(q, rows, m, k):
    """The call's outputs at `rows`, as a call on those rows alone would lay them out."""
    nat = _natural_scales(q["sf"], m, k)
    check_sf(q["sf"], nat, m, (k // 32) * 16)                             # pad rows zero
    at = torch.from_numpy(rows).cuda()
    return dict(codes=q["codes"][at], sf=torch.from_numpy(O.sf_to_mma_layout(np.ascontiguousarray(nat[rows]))).cuda(),
                h=None if q["h"] is None else q["h"][at])


# With 148 SMs: 32, 16 or 8 rows a CTA in three to five rounds; one row a CTA in four or five, 16384 x 5120
# in nine waves of CTAs; two passes a row in three or four rounds.  Ragged last blocks among them.
SHAPES = [(40000, 128), (90000, 128), (29999, 256), (10100, 512), (16300, 384), (5000, 1920), (16384, 5120),
          (2500, 8192), (1300, 8320), (700, 20480)]


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("m,k", SHAPES)
def test_rows_of_every_round(lib, fmt, m, k):
    norm = getattr(lib, "svdq_rmsnorm_" + fmt)
    x, r = _randn(m, k, m + k), _randn(m, k, m + k + 1, 2.0)
    w = (1 + 0.2 * torch.randn(k, device="cuda", generator=torch.Generator(device="cuda").manual_seed(k))).to(
        torch.bfloat16 if fmt == "mxfp8" else torch.float32)
    q = norm(x, w, r)
    assert torch.equal(q["h"], (x.float() + r.float()).to(torch.bfloat16))
    nat = _natural_scales(q["sf"], m, k)
    for a in range(0, m, 128):
        b = min(a + 128, m)
        part = norm(x[a:b], w, r[a:b])
        assert torch.equal(part["codes"], q["codes"][a:b]), f"codes of rows {a}..{b - 1}"
        assert np.array_equal(_natural_scales(part["sf"], b - a, k), nat[a:b]), f"scales of rows {a}..{b - 1}"
    rows = np.unique(np.concatenate([[0, m // 2, m - 2, m - 1], np.random.default_rng(m).choice(m, 24)]))
    xb, rb = host_bits(x[torch.from_numpy(rows).cuda()]), host_bits(r[torch.from_numpy(rows).cuda()])
    _check_norm(_sampled(q, rows, m, k), xb, w.float().cpu().numpy(), rb, 1e-6, fmt)
    plain = norm(x, w, eps=1e-5)                                           # no residual
    assert plain["h"] is None
    _check_norm(_sampled(plain, rows, m, k), xb, w.float().cpu().numpy(), None, 1e-5, fmt)
    # the sum in place of one of its terms, while the next row of both is being loaded
    for which in (0, 1):
        terms = [x.clone(), r.clone()]
        buf = dict(codes=torch.empty_like(q["codes"]), sf=torch.empty_like(q["sf"]), h=terms[which])
        norm(terms[0], w, terms[1], out=buf)
        for key in ("codes", "sf", "h"):
            assert torch.equal(buf[key], q[key]), f"{key} with h in place of {'xr'[which]}"
        assert torch.equal(terms[1 - which], (x, r)[1 - which])
    assert lib.svdq_device_error() == 0
