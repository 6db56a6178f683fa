"""MXFP4 quantiser, read-back and linear, and the RMS norms into MXFP8 and MXFP4,
on the GPU against the oracle in 64 bits (readings R20, R21).

bf16 inputs scale exactly, so the quantiser's codes and scale bytes are compared bit
for bit.  The norm's y carries at most three fp32 roundings (rstd, two products), each
2^-24 relative, so its codes must lie between the encodings of y (1 - 2^-22) and
y (1 + 2^-22).  The linear is held to one bf16 rounding (2^-8 of the value) plus the
accumulation bound of K / 64 fp32 additions per output.
"""
import numpy as np
import pytest
import torch

import synthetic as S
from oracle import svdq_oracle as O
from gpu_util import check_sf, dev_bits, host_bits, requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]

FMT_BITS = {"mxfp8": 1, "mxfp4": 2}                           # codes per byte


@pytest.fixture(scope="module")
def lib():
    import bit_w4a4_quantized_svdq_b200 as P
    return P


def _x(m, k, seed, std=1.0):
    x = S.bf16_bits_to_f32(S.random_bf16((m, k), seed, std)).astype(np.float32)
    rng = np.random.default_rng(seed)
    if m > 3 and k >= 128:
        x[0, :32] = 0.0                                       # an all-zero block
        x[1, 32:64] *= np.float32(2.0 ** 100)                 # large exponents
        x[2, 64:96] *= np.float32(2.0 ** -130)                # subnormal block maximum: scale byte 0
        x[3, :] = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -7.5, -0.25, -0.0], size=k)   # ties, saturation
    return S.f32_to_bf16_bits(x)


def _codes(t, fmt):
    c = t.cpu().numpy()
    return O.unpack_codes(c) if fmt == "mxfp4" else c


def _values(codes, fmt):
    return O.e2m1_decode(codes).astype(np.float64) if fmt == "mxfp4" else O.e4m3_decode(codes).astype(np.float64)


def _natural_scales(sf, m, k):
    return O.sf_from_mma_layout(sf.cpu().numpy(), m, (k // 32) * 16)


def _check_exact(q, x_bits, fmt="mxfp4"):
    m, k = x_bits.shape
    codes, sc = O.mx_quantize_values(O.bf16_to_f64(x_bits), fmt)
    mism = np.argwhere(_codes(q["codes"], fmt) != codes)
    assert mism.size == 0, f"{len(mism)} code mismatches, first {mism[:4].tolist()}"
    check_sf(q["sf"], sc, m, (k // 32) * 16)
    return codes, sc


# ------------------------------------------------------------------------------------------ quantiser
@pytest.mark.parametrize("m,k", [(1, 128), (7, 256), (300, 640), (129, 384), (128, 1920), (4096, 5120)])
def test_quantize_matches_oracle(lib, m, k):
    x_bits = _x(m, k, m + k)
    _check_exact(lib.svdq_quantize_mxfp4(dev_bits(x_bits)), x_bits)
    assert lib.svdq_device_error() == 0


@pytest.mark.parametrize("offset,width", [(0, 1024), (8, 1024), (16, 1040), (24, 776 + 24)])
def test_quantize_strided_rows_and_alignment(lib, offset, width):
    x_bits = _x(200, 768, 9)
    wide = torch.zeros((200, width), dtype=torch.int16, device="cuda")
    wide[:, offset:offset + 768] = dev_bits(x_bits)
    _check_exact(lib.svdq_quantize_mxfp4(wide[:, offset:offset + 768]), x_bits)


def test_quantize_infinities_and_nan(lib):
    x_bits = _x(40, 256, 21)
    f = S.bf16_bits_to_f32(x_bits).copy()
    f[5, 3] = np.inf
    f[6, 40] = -np.inf
    f[7, 200] = np.nan
    f[8, 0:32] = np.nan
    x_bits = S.f32_to_bf16_bits(f)
    codes, sc = _check_exact(lib.svdq_quantize_mxfp4(dev_bits(x_bits)), x_bits)
    assert sc[5, 0] == 255 and sc[6, 1] == 255 and sc[7, 6] == 255 and sc[8, 0] == 255 and (sc == 255).sum() == 4


def test_offsets_past_32_bits(lib):
    """More than 2^31 elements: the last rows equal the same rows quantised alone."""
    m, k = 110000, 20480
    x = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
    tail = torch.randn((128, k), device="cuda").to(torch.bfloat16)
    x[m - 128:] = tail                                       # 110000 % 128 = 48: rows of two row blocks
    q = lib.svdq_quantize_mxfp4(x)
    alone = lib.svdq_quantize_mxfp4(tail)
    assert torch.equal(q["codes"][m - 128:], alone["codes"]) and not q["codes"][:4].any()
    y = lib.svdq_dequantize_mxfp4(q["codes"], q["sf"])
    assert torch.equal(y[m - 128:], lib.svdq_dequantize_mxfp4(alone["codes"], alone["sf"]))
    del x, y, q
    torch.cuda.empty_cache()


# ------------------------------------------------------------------------------------------ read-back
@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("m,k", [(1, 128), (33, 384), (300, 640), (129, 5120)])
def test_dequantize_matches_oracle(lib, fmt, m, k):
    rng = np.random.default_rng(m * k)
    per = FMT_BITS[fmt]
    raw = rng.integers(0, 256, (m, k // per), dtype=np.uint8)
    if fmt == "mxfp8":
        raw[(raw & 0x7F) == 0x7F] = 0x7E                      # no NaN codes here
    sc = rng.integers(100, 150, (m, k // 32), dtype=np.uint8)
    sc[0, 0], sc[0, 1], sc[0, 2], sc[0, 3] = 0, 1, 254, 255   # subnormal and largest scales, NaN
    codes = O.unpack_codes(raw) if fmt == "mxfp4" else raw
    s = np.where(sc == 255, np.nan, np.exp2(sc.astype(np.float64) - 127.0))
    with np.errstate(over="ignore"):
        want = O.f64_to_bf16((_values(codes, fmt).reshape(m, k // 32, 32) * s[:, :, None]).reshape(m, k))
    sf = torch.from_numpy(O.sf_to_mma_layout(sc)).cuda()
    y = lib.svdq_dequantize_mxfp4(torch.from_numpy(raw).cuda(), sf) if fmt == "mxfp4" else \
        lib.svdq_dequantize_mxfp8(torch.from_numpy(raw).cuda(), sf)
    got, w = O.bf16_to_f64(host_bits(y)), O.bf16_to_f64(want)
    assert np.array_equal(np.isnan(got), np.isnan(w)) and np.isnan(w[0, 96:128]).all()
    ok = ~np.isnan(w)
    assert np.array_equal(got[ok], w[ok])


def test_dequantize_e4m3_nan_codes_and_strided_output(lib):
    raw = np.zeros((4, 128), np.uint8)
    raw[1, 5], raw[2, 7] = 0x7F, 0xFF
    sf = torch.from_numpy(O.sf_to_mma_layout(np.full((4, 4), 127, np.uint8))).cuda()
    wide = torch.full((6, 152), 7.0, dtype=torch.bfloat16, device="cuda")
    y = lib.svdq_dequantize_mxfp8(torch.from_numpy(raw).cuda(), sf, out=wide[1:5, 8:136])
    v = y.float().cpu().numpy()
    assert np.isnan(v[1, 5]) and np.isnan(v[2, 7]) and np.isnan(v).sum() == 2
    wide[1:5, 8:136] = 7.0
    assert bool((wide == 7.0).all())                          # nothing around the view was written


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
def test_round_trip_of_representable_values(lib, fmt):
    """Values a format represents come back bit for bit, and quantise to the same codes again."""
    x_bits = _x(257, 640, 5)
    quant = getattr(lib, "svdq_quantize_" + fmt)
    back = getattr(lib, "svdq_dequantize_" + fmt)
    q = quant(dev_bits(x_bits))
    y = back(q["codes"], q["sf"])
    q2 = quant(y)
    y2 = back(q2["codes"], q2["sf"])
    assert torch.equal(y.view(torch.int16), y2.view(torch.int16))


# ------------------------------------------------------------------------------------------ linear
def _check_linear(y, a, w, bias_bits):
    """a, w: fp64 operand values.  One rounding to bf16 and K / 64 + 8 fp32 additions of exact
    products (each at most one unit of 2^-23, the tensor core truncates): per element."""
    y64 = a @ w.T
    if bias_bits is not None:
        y64 = y64 + O.bf16_to_f64(bias_bits)[None, :]
    mag = np.abs(a) @ np.abs(w).T + (0 if bias_bits is None else np.abs(O.bf16_to_f64(bias_bits))[None, :])
    bound = np.abs(y64) * 2.0 ** -8 * (1 + 2.0 ** -8) + (a.shape[1] / 64 + 8) * 2.0 ** -23 * mag + 2.0 ** -134
    err = np.abs(O.bf16_to_f64(host_bits(y)) - y64)
    bad = np.argwhere(~(err <= bound))
    assert bad.size == 0, f"{len(bad)} of {err.size} outputs off, first {bad[:4].tolist()}: {err[tuple(bad[0])]}"


def _operands(lib, m, n, k, seed, fmt="mxfp4"):
    x_bits, w_bits = S.random_bf16((m, k), seed, 1.0), S.random_bf16((n, k), seed + 1, 0.02)
    qa, qw = lib.svdq_quantize_mxfp4(dev_bits(x_bits)), lib.svdq_quantize_mxfp4(dev_bits(w_bits))
    a = O.mx4_dequantize(*O.mx_quantize_values(O.bf16_to_f64(x_bits), "mxfp4"))
    w = O.mx4_dequantize(*O.mx_quantize_values(O.bf16_to_f64(w_bits), "mxfp4"))
    return qa, qw, a, w


LINEAR_SHAPES = [(1, 128, 128), (1, 8, 256), (1, 5120, 5120), (2, 136, 384), (7, 256, 640), (8, 128, 2048),
                 (9, 1160, 1920), (16, 384, 1024), (17, 256, 128), (29, 1280, 5120), (32, 128, 256), (33, 264, 640),
                 (64, 512, 1024), (65, 128, 384), (115, 640, 1280), (128, 256, 512), (129, 392, 640), (255, 512, 256),
                 (256, 256, 128), (257, 520, 1152), (300, 512, 640), (515, 1160, 1920), (1000, 768, 1024),
                 (1024, 2560, 256), (2050, 136, 512), (513, 5000, 256), (512, 5120, 1152), (1800, 2200, 384),
                 (2304, 2304, 128), (300, 8, 128), (1000, 24, 256), (5, 50000, 256), (2, 136, 65536), (300, 264, 32768),
                 (100, 264, 4096), (100, 264, 4224), (60, 20000, 512), (128, 20000, 4352), (16, 1160, 16384)]


@pytest.mark.parametrize("m,n,k", LINEAR_SHAPES)
def test_linear_matches_oracle(lib, m, n, k):
    qa, qw, a, w = _operands(lib, m, n, k, 3 * m + n + k)
    bias = S.random_bf16((n,), 7, 0.05)
    args = (qa["codes"], qa["sf"], qw["codes"], qw["sf"])
    _check_linear(lib.svdq_linear_mxfp4(*args, dev_bits(bias)), a, w, bias)
    _check_linear(lib.svdq_linear_mxfp4(*args), a, w, None)
    assert lib.svdq_device_error() == 0


@pytest.mark.parametrize("m,n,k", [(3, 136, 256), (40, 264, 384), (200, 392, 640), (700, 520, 512)])
def test_linear_writes_only_its_output(lib, m, n, k):
    qa, qw, a, w = _operands(lib, m, n, k, 17)
    wide = torch.full((m + 3, n + 24), 5.0, dtype=torch.bfloat16, device="cuda")
    out = wide[1:m + 1, 8:n + 8]
    y = lib.svdq_linear_mxfp4(qa["codes"], qa["sf"], qw["codes"], qw["sf"], None, out=out)
    assert y.data_ptr() == out.data_ptr()
    _check_linear(y.contiguous(), a, w, None)
    out.fill_(5.0)
    assert bool((wide == 5.0).all())


@pytest.mark.parametrize("m", [1, 40, 300])
def test_linear_wide_exponents(lib, m):
    """Rows and columns of very different scale, zero blocks among them: products from 2^-100 to 2^100."""
    n, k = 264, 640
    rng = np.random.default_rng(m)
    x = rng.standard_normal((m, k)) * np.exp2(rng.integers(-60, 60, (m, 1)))
    w = rng.standard_normal((n, k)) * np.exp2(rng.integers(-40, 40, (n, 1)))
    x[:, 32:64] = 0.0
    w[::3, 96:160] = 0.0
    x_bits, w_bits = O.f64_to_bf16(x), O.f64_to_bf16(w)
    qa, qw = lib.svdq_quantize_mxfp4(dev_bits(x_bits)), lib.svdq_quantize_mxfp4(dev_bits(w_bits))
    a = O.mx4_dequantize(*O.mx_quantize_values(O.bf16_to_f64(x_bits), "mxfp4"))
    b = O.mx4_dequantize(*O.mx_quantize_values(O.bf16_to_f64(w_bits), "mxfp4"))
    _check_linear(lib.svdq_linear_mxfp4(qa["codes"], qa["sf"], qw["codes"], qw["sf"]), a, b, None)


@pytest.mark.parametrize("m", [1, 20, 300])
def test_linear_nan_scales_reach_their_rows_and_columns_only(lib, m):
    n, k = 256, 512
    x_bits, w_bits = S.random_bf16((m, k), 1, 1.0), S.random_bf16((n, k), 2, 0.02)
    f = S.bf16_bits_to_f32(w_bits).copy()
    f[5, 100] = np.nan
    qa, qw = lib.svdq_quantize_mxfp4(dev_bits(x_bits)), lib.svdq_quantize_mxfp4(dev_bits(S.f32_to_bf16_bits(f)))
    y = lib.svdq_linear_mxfp4(qa["codes"], qa["sf"], qw["codes"], qw["sf"]).float()
    nan = torch.isnan(y)
    assert bool(nan[:, 5].all()) and int(nan.sum()) == m


@pytest.mark.parametrize("m,n,k", [(1, 5120, 5120), (29, 2560, 2560), (2048, 2560, 128), (4000, 1280, 384)])
def test_linear_repeatable(lib, m, n, k):
    qa, qw, _, _ = _operands(lib, m, n, k, 91)
    args = (qa["codes"], qa["sf"], qw["codes"], qw["sf"])
    y0 = lib.svdq_linear_mxfp4(*args)
    for _ in range(20):
        assert torch.equal(lib.svdq_linear_mxfp4(*args).view(torch.int16), y0.view(torch.int16))
    assert lib.svdq_device_error() == 0


def test_linear_large_sampled(lib):
    """The attention projection's shape; the oracle on sampled rows, every column."""
    L = S.make_layer(1)
    qa, qw = lib.svdq_quantize_mxfp4(dev_bits(L.x)), lib.svdq_quantize_mxfp4(dev_bits(L.w))
    y = lib.svdq_linear_mxfp4(qa["codes"], qa["sf"], qw["codes"], qw["sf"], dev_bits(L.bias))
    rows = np.random.default_rng(0).choice(L.x.shape[0], 96, replace=False)
    a = O.mx4_dequantize(*O.mx_quantize_values(O.bf16_to_f64(L.x[rows]), "mxfp4"))
    w = O.mx4_dequantize(*O.mx_quantize_values(O.bf16_to_f64(L.w), "mxfp4"))
    _check_linear(y[torch.from_numpy(rows).cuda()].contiguous(), a, w, L.bias)


# Several tiles per pair of CTAs, 1 to 5 ring slots a tile, and each tile width: 256, 192 and 128 columns.
@pytest.mark.parametrize("m,n,k", [(4096, 15360, 256), (4000, 15352, 1152), (4096, 5120, 384), (4097, 5112, 128),
                                   (3000, 9472, 640), (8192, 3712, 256), (2500, 3840, 1408), (16300, 128, 256)])
def test_linear_many_tiles_sampled(lib, m, n, k):
    x_bits, w_bits = S.random_bf16((m, k), m, 1.0), S.random_bf16((n, k), n, 0.02)
    bias = S.random_bf16((n,), 7, 0.05)
    qa, qw = lib.svdq_quantize_mxfp4(dev_bits(x_bits)), lib.svdq_quantize_mxfp4(dev_bits(w_bits))
    y = lib.svdq_linear_mxfp4(qa["codes"], qa["sf"], qw["codes"], qw["sf"], dev_bits(bias))
    rows = np.sort(np.random.default_rng(1).choice(m, 160, replace=False))
    rows[-1] = m - 1
    a = O.mx4_dequantize(*O.mx_quantize_values(O.bf16_to_f64(x_bits[rows]), "mxfp4"))
    w = O.mx4_dequantize(*O.mx_quantize_values(O.bf16_to_f64(w_bits), "mxfp4"))
    _check_linear(y[torch.from_numpy(rows).cuda()].contiguous(), a, w, bias)
    for _ in range(5):
        again = lib.svdq_linear_mxfp4(qa["codes"], qa["sf"], qw["codes"], qw["sf"], dev_bits(bias))
        assert torch.equal(again.view(torch.int16), y.view(torch.int16))
    assert lib.svdq_device_error() == 0


# ------------------------------------------------------------------------------------------ norms
def _check_norm(q, x_bits, weight, res_bits, eps, fmt):
    m, k = x_bits.shape
    h_bits, y = O.rmsnorm(x_bits, weight, res_bits, eps)
    if res_bits is None:
        assert q["h"] is None
    else:
        assert np.array_equal(host_bits(q["h"]), h_bits)
    got = _natural_scales(q["sf"], m, k).astype(np.int64)
    d = 2.0 ** -22
    amax = np.abs(y).reshape(m, k // 32, 32).max(axis=2)
    emax = 8 if fmt == "mxfp8" else 2
    lo, hi = O.mx_format_exponent(amax * (1 - d), emax) + 127, O.mx_format_exponent(amax * (1 + d), emax) + 127
    assert ((got >= lo) & (got <= hi)).all(), "scale bytes"
    check_sf(q["sf"], got.astype(np.uint8), m, (k // 32) * 16)          # pad rows zero
    s = (y.reshape(m, k // 32, 32) * np.exp2(127.0 - got)[:, :, None]).reshape(m, k)
    enc = (lambda v: _values(O.e2m1_encode(v), fmt)) if fmt == "mxfp4" else (lambda v: _values(O.e4m3_encode(v), fmt))
    a, b = enc(s * (1 - d)), enc(s * (1 + d))
    v = _values(_codes(q["codes"], fmt), fmt)
    bad = np.argwhere((v < np.minimum(a, b)) | (v > np.maximum(a, b)))
    assert bad.size == 0, f"{len(bad)} codes outside their interval, first {bad[:4].tolist()}"
    assert (v == enc(s)).mean() > 0.999


NORM_SHAPES = [(1, 128), (5, 128), (130, 128), (3, 256), (300, 384), (64, 512), (129, 640), (1, 1920), (1037, 1920),
               (200, 5120), (1, 8192), (40, 8320), (17, 16384), (9, 20480), (130, 32768), (3, 40960)]


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("m,k", NORM_SHAPES)
def test_norm_matches_oracle(lib, fmt, m, k):
    x_bits, r_bits = S.random_bf16((m, k), m + k, 1.0), S.random_bf16((m, k), m + k + 1, 3.0)
    w = (1.0 + 0.2 * np.random.default_rng(k).standard_normal(k)).astype(np.float32)
    w_bits = S.f32_to_bf16_bits(w)
    norm = getattr(lib, "svdq_rmsnorm_" + fmt)
    # bf16 weight with a residual, fp32 weight without one
    _check_norm(norm(dev_bits(x_bits), dev_bits(w_bits).view(torch.bfloat16), dev_bits(r_bits)), x_bits,
                S.bf16_bits_to_f32(w_bits), r_bits, 1e-6, fmt)
    _check_norm(norm(dev_bits(x_bits), torch.from_numpy(w).cuda(), eps=1e-5), x_bits, w, None, 1e-5, fmt)
    assert lib.svdq_device_error() == 0


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_norm_strides_alignment_and_in_place(lib, fmt):
    m, k = 77, 640
    x_bits, r_bits = S.random_bf16((m, k), 1, 1.0), S.random_bf16((m, k), 2, 1.0)
    w = np.linspace(0.5, 1.5, k).astype(np.float32)
    norm = getattr(lib, "svdq_rmsnorm_" + fmt)
    for off in (0, 8, 16):                                    # 32-byte aligned rows and not
        wx = torch.zeros((m, k + 40), dtype=torch.int16, device="cuda")
        wr, wh = wx.clone(), torch.full((m + 1, k + 40), 3.0, dtype=torch.bfloat16, device="cuda")
        wx[:, off:off + k], wr[:, 8:8 + k] = dev_bits(x_bits), dev_bits(r_bits)
        out = lib.svdq_quantize_mxfp8(wx[:, off:off + k]) if fmt == "mxfp8" else lib.svdq_quantize_mxfp4(wx[:, off:off + k])
        q = norm(wx[:, off:off + k], torch.from_numpy(w).cuda(), wr[:, 8:8 + k], out=dict(out, h=wh[:m, off:off + k]))
        assert q["h"].data_ptr() == wh[:m, off:off + k].data_ptr() and q["codes"].data_ptr() == out["codes"].data_ptr()
        _check_norm(dict(q, h=q["h"].contiguous()), x_bits, w, r_bits, 1e-6, fmt)
        wh[:m, off:off + k] = 3.0
        assert bool((wh == 3.0).all())
    for which in ("x", "r"):                                  # the sum replaces one of its terms
        x, r = dev_bits(x_bits).view(torch.bfloat16), dev_bits(r_bits).view(torch.bfloat16)
        h = x if which == "x" else r
        first = norm(x.clone(), torch.from_numpy(w).cuda(), r.clone())
        buf = getattr(lib, "svdq_quantize_" + fmt)(x)
        q = norm(x, torch.from_numpy(w).cuda(), r, out=dict(buf, h=h))
        assert torch.equal(h, first["h"]) and torch.equal(q["codes"], first["codes"]) and torch.equal(q["sf"], first["sf"])


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("k", [256, 640, 10240])
def test_norm_rows_of_zeros_extremes_and_nan(lib, fmt, k):
    m = 9
    f = S.bf16_bits_to_f32(S.random_bf16((m, k), 3, 1.0)).copy()
    f[1] = 0.0                                                # rstd = 1 / sqrt(eps), y = 0
    f[2] = np.where(np.arange(k) % 2, 3e38, -3e38)            # squares past fp32
    f[3] *= np.float32(1e-38)                                 # squares below fp32: eps decides
    f[5, 7] = np.nan
    f[6, 9] = np.inf
    x_bits = S.f32_to_bf16_bits(f)
    w = np.ones(k, np.float32)
    q = getattr(lib, "svdq_rmsnorm_" + fmt)(dev_bits(x_bits), torch.from_numpy(w).cuda())
    v = getattr(lib, "svdq_dequantize_" + fmt)(q["codes"], q["sf"]).double().cpu().numpy()
    assert not v[1].any()
    good = [0, 1, 2, 3, 4, 7, 8]
    _, y = O.rmsnorm(x_bits[good], w, None, 1e-6)
    step = 2.0 ** -4 if fmt == "mxfp8" else 2.0 ** -2          # half a step of the format, relative to the block's top
    top = np.abs(y).reshape(len(good), -1, 32).max(axis=2).repeat(32, axis=1)
    assert (np.abs(v[good] - y) <= 2 * step * top).all()
    assert np.isnan(v[5]).all()                                # NaN spreads over its row
    assert np.isnan(v[6, 9])                                   # inf / inf; in mxfp4 its block with it
    rest = np.ones(k, bool)
    rest[0:32] = False
    assert not v[6, rest].any()                                # finite / inf


def test_norm_codes_do_not_depend_on_the_rows_beside_them(lib):
    """A row's codes are the same whatever launch shape it is part of."""
    x = torch.randn((2000, 1920), device="cuda").to(torch.bfloat16)
    w = torch.randn(1920, device="cuda")
    full = lib.svdq_rmsnorm_mxfp8(x, w)
    for r in (0, 777, 1999):
        assert torch.equal(lib.svdq_rmsnorm_mxfp8(x[r:r + 1], w)["codes"][0], full["codes"][r])


# ------------------------------------------------------------------------------------------ together
def _block(lib, s, fmt="mxfp4", out=None, stream=None):
    """A pre-norm block's entry as a program runs it: residual and norm, the projection, and the
    projection's output normed again against the carried sum."""
    kw = {} if stream is None else dict(stream=stream)
    q = getattr(lib, "svdq_rmsnorm_" + fmt)(s["x"], s["g1"], s["r"], **kw)
    y = getattr(lib, "svdq_linear_" + fmt)(q["codes"], q["sf"], s["w"]["codes"], s["w"]["sf"], s["b"], **kw)
    q2 = lib.svdq_rmsnorm_mxfp4(y, s["g2"], q["h"], **kw)
    z = lib.svdq_linear_mxfp4(q2["codes"], q2["sf"], s["w4"]["codes"], s["w4"]["sf"], None, **kw)
    return q["h"], y, q2["h"], z


def _block_state(lib, m, k, seed, fmt="mxfp4"):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    w = (0.02 * rnd(k, k)).to(torch.bfloat16)
    return dict(x=rnd(m, k).to(torch.bfloat16), r=(3 * rnd(m, k)).to(torch.bfloat16), g1=1 + 0.1 * rnd(k),
                g2=(1 + 0.1 * rnd(k)).to(torch.bfloat16), b=(0.02 * rnd(k)).to(torch.bfloat16),
                w=getattr(lib, "svdq_quantize_" + fmt)(w), w4=lib.svdq_quantize_mxfp4(w))


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("m", [1, 29, 700])
def test_block_run_together_matches_oracle(lib, fmt, m):
    k = 640
    s = _block_state(lib, m, k, m, fmt)
    h1, y, h2, z = _block(lib, s, fmt)
    bits = lambda t: host_bits(t)  # noqa: E731
    w = getattr(lib, "svdq_dequantize_" + fmt)(s["w"]["codes"], s["w"]["sf"]).double().cpu().numpy()
    w4 = lib.svdq_dequantize_mxfp4(s["w4"]["codes"], s["w4"]["sf"]).double().cpu().numpy()
    h_bits, _ = O.rmsnorm(bits(s["x"]), s["g1"].cpu().numpy(), bits(s["r"]), 1e-6)
    assert np.array_equal(bits(h1), h_bits)
    q = getattr(lib, "svdq_rmsnorm_" + fmt)(s["x"], s["g1"], s["r"])
    a = getattr(lib, "svdq_dequantize_" + fmt)(q["codes"], q["sf"]).double().cpu().numpy()
    y64 = a @ w.T + s["b"].double().cpu().numpy()[None, :]
    # MXFP8 takes K / 32 additions, MXFP4 K / 64: the larger for both
    bound = np.abs(y64) * 2.0 ** -8 * (1 + 2.0 ** -8) + (k / 32 + 8) * 2.0 ** -23 * (np.abs(a) @ np.abs(w).T + 1)
    assert (np.abs(y.double().cpu().numpy() - y64) <= bound).all()
    q2 = lib.svdq_rmsnorm_mxfp4(y, s["g2"], h1)
    _check_norm(q2, bits(y), s["g2"].float().cpu().numpy(), bits(h1), 1e-6, "mxfp4")
    assert torch.equal(q2["h"], h2)
    _check_linear(z, lib.svdq_dequantize_mxfp4(q2["codes"], q2["sf"]).double().cpu().numpy(), w4, None)


@pytest.mark.parametrize("m", [1, 29, 300])
def test_block_captured_and_replayed(lib, m):
    s = _block_state(lib, m, 1280, 40 + m)
    want = [t.clone() for t in _block(lib, s)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):                                         # two graphs of the same tensors
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_block(lib, s))
        graphs.append(g)
    new_x = torch.randn_like(s["x"])
    old_x = s["x"].clone()
    for g, o in zip(graphs, outs):
        for x in (new_x, old_x):
            s["x"].copy_(x)
            g.replay()
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(o, want))
    s["x"].copy_(new_x)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], _block(lib, s)))


def test_two_streams_at_once(lib):
    states = [_block_state(lib, m, 1280, 70 + m) for m in (1, 40, 300, 3)]
    want = [[t.clone() for t in _block(lib, s)] for s in states]
    streams = [torch.cuda.Stream() for _ in states]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        got = [_block(lib, s, stream=st) for s, st in zip(states, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w))
    assert lib.svdq_device_error() == 0


def test_two_host_threads(lib):
    """Calls from two threads at once, each on a stream of its own (the binding releases the interpreter
    lock inside the library)."""
    import threading
    states = [_block_state(lib, m, 1280, 170 + m) for m in (2, 300)]
    want = [[t.clone() for t in _block(lib, s)] for s in states]
    torch.cuda.synchronize()
    bad = []

    def work(s, w):
        st = torch.cuda.Stream()
        for _ in range(30):
            got = _block(lib, s, stream=st)
            st.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, w)):
                bad.append(1)

    threads = [threading.Thread(target=work, args=a) for a in zip(states, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and lib.svdq_device_error() == 0


def test_refusals_on_the_device(lib):
    """Views the kernels cannot take are refused, and the next call runs."""
    x = torch.zeros((4, 264), dtype=torch.bfloat16, device="cuda")
    q = lib.svdq_quantize_mxfp4(x[:, :256])
    with pytest.raises(lib.SvdqError) as e:
        lib.svdq_quantize_mxfp4(x[:, 4:260])                  # rows not 16-byte aligned
    assert e.value.status == lib._lib.SVDQ_ERR_MISALIGNED
    with pytest.raises(ValueError):
        lib.svdq_quantize_mxfp4(x.t()[:128])                  # columns not adjacent
    with pytest.raises(lib.SvdqError):
        lib.svdq_linear_mxfp4(q["codes"][:0], q["sf"], q["codes"], q["sf"])
    with pytest.raises(lib.SvdqError) as e:
        lib.svdq_linear_mxfp4(q["codes"], q["sf"], q["codes"], q["sf"])      # N = 4
    assert e.value.status == lib._lib.SVDQ_ERR_UNSUPPORTED
    with pytest.raises(lib.SvdqError):
        lib.svdq_rmsnorm_mxfp8(x[:, :256], torch.ones(256, device="cuda"), eps=0.0)
    with pytest.raises(ValueError, match="different devices"):
        lib.svdq_rmsnorm_mxfp8(x[:, :256], torch.ones(256))
    _check_exact(lib.svdq_quantize_mxfp4(x[:, :256]), host_bits(x[:, :256].contiguous()))
