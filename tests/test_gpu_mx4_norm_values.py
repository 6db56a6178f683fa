"""Values at the ends of the norms' range, and what a round trip leaves: code by code.

y = h * rstd * weight carries a rounding of rstd and of two products.  Each is 2^-24 relative,
except rstd's where it is subnormal: half of fp32's smallest step, 2^-150, against the rstd of a row
of +-3e38, 2^-128 < 1 / 3e38, is 2^-22.  Together less than 2^-21."""
import numpy as np
import pytest
import torch

import synthetic as S
from oracle import svdq_oracle as O
from gpu_util import dev_bits, requires_cuda
from test_gpu_mx4 import _codes, _natural_scales, _values, _x

pytestmark = [pytest.mark.gpu, requires_cuda]

D = 2.0 ** -21


@pytest.fixture(scope="module")
def lib():
    import bit_w4a4_quantized_svdq_b200 as P
    return P


def _encode(v, fmt):
    return _values(O.e2m1_encode(v) if fmt == "mxfp4" else O.e4m3_encode(v), fmt)


def _check_rows(q, y, rows, m, k, fmt):
    """Scale bytes and codes of `rows` between those of y (1 - D) and y (1 + D); y: fp64 of those rows."""
    got = _natural_scales(q["sf"], m, k).astype(np.int64)[rows]
    amax = np.abs(y).reshape(len(rows), k // 32, 32).max(axis=2)
    emax = 8 if fmt == "mxfp8" else 2
    lo, hi = (O.mx_format_exponent(amax * f, emax) + 127 for f in (1 - D, 1 + D))
    assert ((got >= lo) & (got <= hi)).all()
    s = (y.reshape(len(rows), k // 32, 32) * np.exp2(127.0 - got)[:, :, None]).reshape(len(rows), k)
    a, b = _encode(s * (1 - D), fmt), _encode(s * (1 + D), fmt)
    v = _values(_codes(q["codes"], fmt)[rows], fmt)
    bad = np.argwhere((v < np.minimum(a, b)) | (v > np.maximum(a, b)))
    assert bad.size == 0, f"{len(bad)} codes outside their interval, first {bad[:4].tolist()}"


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("k", [128, 256, 640, 10240])
def test_rows_whose_squares_leave_fp32(lib, fmt, k):
    m = 9
    f = S.bf16_bits_to_f32(S.random_bf16((m, k), 3, 1.0)).copy()
    f[1] = 0.0                                                # rstd = 1 / sqrt(eps), y = 0
    f[2] = np.where(np.arange(k) % 2, 3e38, -3e38)            # squares past fp32: y = +-1
    f[3] *= np.float32(1e-38)                                 # squares below fp32: eps decides
    f[4] *= np.float32(1e18)                                  # past the range of the fast reciprocal root
    f[5, 7] = np.nan                                          # rows beside a NaN and an infinity
    f[6, 9] = np.inf
    f[7] *= np.float32(1e-3)                                  # squares beside eps
    x_bits = S.f32_to_bf16_bits(f)
    rows = [0, 1, 2, 3, 4, 7, 8]
    for eps in (1e-6, 1e-38):                                 # the second below the fast root's range too
        q = getattr(lib, "svdq_rmsnorm_" + fmt)(dev_bits(x_bits), torch.ones(k, device="cuda"), eps=eps)
        _, y = O.rmsnorm(x_bits[rows], np.ones(k, np.float32), None, eps)
        _check_rows(q, y, rows, m, k, fmt)
        v = getattr(lib, "svdq_dequantize_" + fmt)(q["codes"], q["sf"]).double().cpu().numpy()
        assert not v[1].any()


@pytest.mark.parametrize("k", [256, 640, 10240])
def test_product_past_fp32(lib, k):
    """h rstd weight past fp32's range, or an infinite weight.  MXFP4 gives the block the NaN scale.
    MXFP8 gives it the largest scale, 2^120, and the element the largest code, +-448: as a value past
    fp32 too, so it reads back as an infinity.  Other blocks are as without it."""
    m = 5
    x_bits = S.random_bf16((m, k), 5, 1.0)
    f = S.bf16_bits_to_f32(x_bits).copy()
    f[:, 3], f[:, 70], f[:, 100] = [4.0, -4.0, 4.0, 4.0, -4.0], [2.0, 2.0, -2.0, 2.0, 2.0], 1.0
    f[:, 71] = 0.0
    x_bits = S.f32_to_bf16_bits(f)
    w = np.ones(k, np.float32)
    w[3], w[70], w[100] = 3e38, np.inf, 1e37                  # 4 rstd 3e38 overflows, 1 rstd 1e37 does not
    args = dev_bits(x_bits), torch.from_numpy(w).cuda()
    _, y = O.rmsnorm(x_bits, np.where(np.isin(np.arange(k), [3, 70]), 0.0, w), None, 1e-6)

    q = lib.svdq_rmsnorm_mxfp4(*args)
    sc, codes = _natural_scales(q["sf"], m, k), _codes(q["codes"], "mxfp4")
    assert (sc[:, [0, 2]] == 255).all() and (sc == 255).sum() == 2 * m
    assert not codes[:, 0:32].any() and not codes[:, 64:96].any()
    v = lib.svdq_dequantize_mxfp4(q["codes"], q["sf"]).float().cpu().numpy()
    assert np.isnan(v[:, 0:32]).all() and np.isnan(v[:, 64:96]).all() and np.isnan(v).sum() == 64 * m

    q = lib.svdq_rmsnorm_mxfp8(*args)
    sc, codes = _natural_scales(q["sf"], m, k), _codes(q["codes"], "mxfp8")
    assert (sc[:, [0, 2]] == 247).all() and (sc == 247).sum() == 2 * m
    neg = np.signbit(f)
    for c in (3, 70):
        assert (codes[:, c] == np.where(neg[:, c], 0xFE, 0x7E)).all()
    v = lib.svdq_dequantize_mxfp8(q["codes"], q["sf"]).float().cpu().numpy()
    assert np.array_equal(np.argwhere(np.isinf(v)), [[r, c] for r in range(m) for c in (3, 70)])
    assert np.array_equal(np.signbit(v[:, [3, 70]]), neg[:, [3, 70]]) and not np.isnan(v).any()

    for fmt in ("mxfp8", "mxfp4"):                             # the blocks beside them
        q = getattr(lib, "svdq_rmsnorm_" + fmt)(*args)
        got = _natural_scales(q["sf"], m, k).astype(np.int64)
        keep = np.ones(k // 32, bool)
        keep[[0, 2]] = False
        s = (y.reshape(m, -1, 32) * np.exp2(127.0 - got)[:, :, None])[:, keep].reshape(m, -1)
        a, b = _encode(s * (1 - D), fmt), _encode(s * (1 + D), fmt)
        vals = _values(_codes(q["codes"], fmt), fmt).reshape(m, -1, 32)[:, keep].reshape(m, -1)
        assert ((vals >= np.minimum(a, b)) & (vals <= np.maximum(a, b))).all()
    assert lib.svdq_device_error() == 0


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_infinite_weight_on_zero_is_nan(lib, fmt):
    """0 * infinity: a NaN code under MXFP8, a NaN block under MXFP4; the rest of the row is finite."""
    x = torch.ones((3, 256), dtype=torch.bfloat16, device="cuda")
    x[1, 40] = 0.0
    w = torch.full((256,), 1.5, device="cuda")                 # 1.5 is nearest to 1.5 rstd in both formats
    w[40] = float("inf")
    q = getattr(lib, "svdq_rmsnorm_" + fmt)(x, w)
    v = getattr(lib, "svdq_dequantize_" + fmt)(q["codes"], q["sf"]).float()
    assert bool(torch.isnan(v[1, 40]))
    rest = torch.ones(256, dtype=torch.bool, device="cuda")
    rest[32:64] = False
    assert bool((v[:, rest] == 1.5).all())


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_round_trip_gives_the_same_codes(lib, fmt):
    """Quantised, read back and quantised again: the same codes and scale bytes, signs of zeros too.
    (A block's largest code keeps its exponent, and every value here is exact in bf16.)"""
    quant, back = getattr(lib, "svdq_quantize_" + fmt), getattr(lib, "svdq_dequantize_" + fmt)
    q = quant(dev_bits(_x(257, 640, 5)))
    q2 = quant(back(q["codes"], q["sf"]))
    assert torch.equal(q2["codes"], q["codes"]) and torch.equal(q2["sf"], q["sf"])
