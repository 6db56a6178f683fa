"""MXFP4 and the norms into the microscaled formats, on CPU: the oracle's pins, sizes,
refusals of the C ABI and of the binding, and the binding's marshalling."""
import ctypes

import numpy as np
import pytest
import torch

from bit_w4a4_quantized_svdq_b200 import _lib, ops
from oracle import svdq_oracle as O

FAKE = 0x10000          # an aligned non-null "device" pointer; never dereferenced on these paths
INVALID, UNSUPPORTED, MISALIGNED, NO_DEVICE = (_lib.SVDQ_ERR_INVALID_ARG, _lib.SVDQ_ERR_UNSUPPORTED,
                                               _lib.SVDQ_ERR_MISALIGNED, _lib.SVDQ_ERR_NO_DEVICE)


# ---------------------------------------------------------------------------------------------- the oracle
def test_oracle_mxfp4_worked_block():
    b = np.zeros((1, 32))
    b[0, :9] = [6.0, -3.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]        # amax 6: exponent 2 - 2 = 0, scale 1
    codes, sc = O.mx_quantize_values(b, "mxfp4")
    assert sc[0, 0] == 127
    assert codes[0, :9].tolist() == [7, 8 | 5, 0, 2, 2, 4, 4, 6, 6]      # ties to the even code
    codes, sc = O.mx_quantize_values(b * 2.0 ** -20, "mxfp4")
    assert sc[0, 0] == 107 and codes[0, :9].tolist() == [7, 13, 0, 2, 2, 4, 4, 6, 6]
    b[0, 0] = 7.9                                                         # still exponent 0: saturates at 6
    assert O.mx_quantize_values(b, "mxfp4")[0][0, 0] == 7
    b[0, 0] = 8.0                                                         # exponent 1: 8 = 4 * 2
    codes, sc = O.mx_quantize_values(b, "mxfp4")
    assert sc[0, 0] == 128 and codes[0, 0] == 6


def test_oracle_mxfp4_zero_tiny_and_nan_blocks():
    b = np.zeros((4, 32))
    b[1, 3] = 2.0 ** -133                                                 # bf16's least subnormal
    b[2, 3] = np.nan
    b[3, 3] = -np.inf
    codes, sc = O.mx_quantize_values(b, "mxfp4")
    assert sc[:, 0].tolist() == [0, 0, 255, 255] and not codes.any()
    v = O.mx4_dequantize(codes, sc)
    assert not v[:2].any() and np.isnan(v[2:]).all()


def test_oracle_mxfp4_against_exhaustive_search():
    """Every code is a nearest value of the scaled grid; representable blocks are lossless."""
    rng = np.random.default_rng(0)
    x = O.bf16_to_f64(O.f64_to_bf16(rng.standard_normal((50, 64)) * np.exp2(rng.integers(-40, 40, (50, 64)))))
    codes, sc = O.mx_quantize_values(x, "mxfp4")
    v = O.mx4_dequantize(codes, sc)
    grid = np.concatenate([O.E2M1_MAGNITUDES, -O.E2M1_MAGNITUDES]).astype(np.float64)
    s = np.exp2(sc.astype(np.float64) - 127).repeat(32, axis=1)
    best = np.abs(x[:, :, None] - grid * s[:, :, None]).min(axis=2)
    assert np.array_equal(np.abs(x - v), best)
    again = O.mx_quantize_values(v, "mxfp4")
    assert np.array_equal(O.mx4_dequantize(*again), v)


def test_oracle_mx_values_agree_with_the_mxfp8_oracle():
    rng = np.random.default_rng(1)
    bits = O.f64_to_bf16(rng.standard_normal((20, 128)) * np.exp2(rng.integers(-30, 30, (20, 1))))
    a, b = O.mx_quantize(bits), O.mx_quantize_values(O.bf16_to_f64(bits), "mxfp8")
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_oracle_rmsnorm_closed_forms():
    x = O.f64_to_bf16(np.array([[3.0, -4.0] * 64, [0.0] * 128]))
    h, y = O.rmsnorm(x, np.ones(128), None, 1e-30)
    assert np.array_equal(h, x)
    np.testing.assert_allclose(y[0], O.bf16_to_f64(x)[0] / np.sqrt(12.5), rtol=1e-15)
    assert not y[1].any()
    h, y = O.rmsnorm(x, np.full(128, 2.0), x, 1e-30)                      # x + x: y does not change with scale
    assert np.array_equal(O.bf16_to_f64(h), 2 * O.bf16_to_f64(x))
    np.testing.assert_allclose(y[0], 2 * O.bf16_to_f64(x)[0] / np.sqrt(12.5), rtol=1e-15)
    h, _ = O.rmsnorm(O.f64_to_bf16(np.full((1, 32), 1.0)), np.ones(32), O.f64_to_bf16(np.full((1, 32), 2.0 ** -8)), 1e-6)
    assert (O.bf16_to_f64(h) == 1.0).all()                                # the sum is rounded to bf16 (tie to even)


# ------------------------------------------------------------------------------------------- the C ABI
def test_sizes():
    lib = _lib.load()
    assert lib.svdq_mxfp4_sf_bytes(1, 128) == 128 * 4
    assert lib.svdq_mxfp4_sf_bytes(129, 5120) == 256 * 160
    assert lib.svdq_mxfp4_sf_bytes(4, 96) == 0 and lib.svdq_mxfp4_sf_bytes(0, 128) == 0
    for rows in (-1, 0, 1, 127, 128, 129, 5000):
        for k in (-128, 0, 32, 96, 128, 192, 256, 5120):
            assert ops._mx_sf_size(rows, k) == ops.mxfp4_sf_bytes(rows, k) == ops.mxfp8_sf_bytes(rows, k)


def test_quantize_and_dequantize_reject_bad_arguments():
    lib = _lib.load()
    p, z = ctypes.c_void_p(FAKE), ctypes.c_void_p
    for fn in (lib.svdq_quantize_mxfp4, ):
        assert fn(None, 4, 128, 128, p, p, None) == INVALID
        assert fn(p, 4, 128, 128, None, p, None) == INVALID
        assert fn(p, 4, 128, 128, p, None, None) == INVALID
        assert fn(p, 0, 128, 128, p, p, None) == INVALID
        assert fn(p, 4, 0, 128, p, p, None) == INVALID
        assert fn(p, 4, 128, 120, p, p, None) == INVALID                   # ldx < K
        assert fn(p, 4, 192, 192, p, p, None) == UNSUPPORTED               # K % 128
        assert fn(z(FAKE + 8), 4, 128, 128, p, p, None) == MISALIGNED
        assert fn(p, 4, 128, 132, p, p, None) == MISALIGNED                # row stride
        assert fn(p, 4, 128, 128, z(FAKE + 8), p, None) == MISALIGNED
        assert fn(p, 4, 128, 128, p, z(FAKE + 2), None) == MISALIGNED
        assert fn(p, 1 << 39, 1 << 14, 1 << 14, p, p, None) == UNSUPPORTED
        assert fn(p, 4, 128, 128, p, p, None) == NO_DEVICE
    for fn in (lib.svdq_dequantize_mxfp4, lib.svdq_dequantize_mxfp8):
        assert fn(None, p, 4, 128, p, 128, None) == INVALID
        assert fn(p, None, 4, 128, p, 128, None) == INVALID
        assert fn(p, p, 4, 128, None, 128, None) == INVALID
        assert fn(p, p, 0, 128, p, 128, None) == INVALID
        assert fn(p, p, 4, 128, p, 64, None) == INVALID
        assert fn(p, p, 4, 160, p, 160, None) == UNSUPPORTED
        assert fn(z(FAKE + 8), p, 4, 128, p, 128, None) == MISALIGNED
        assert fn(p, p, 4, 128, p, 132, None) == MISALIGNED
        assert fn(p, p, 4, 128, p, 128, None) == NO_DEVICE


def test_linear_rejects_bad_arguments():
    lib = _lib.load()
    p, z = ctypes.c_void_p(FAKE), ctypes.c_void_p
    base = dict(a=p, asf=p, w=p, wsf=p, bias=None, y=p, ldy=256, m=4, n=256, k=128)

    def call(**kw):
        c = dict(base, **kw)
        return lib.svdq_linear_mxfp4(c["a"], c["asf"], c["w"], c["wsf"], c["bias"], c["y"], c["ldy"], c["m"], c["n"],
                                     c["k"], None)

    for name in ("a", "asf", "w", "wsf", "y"):
        assert call(**{name: None}) == INVALID
        assert call(**{name: z(FAKE + 8)}) == MISALIGNED
    assert call(bias=z(FAKE + 2)) == MISALIGNED
    assert call(m=0) == INVALID and call(n=0) == INVALID and call(k=0) == INVALID
    assert call(ldy=248) == INVALID
    assert call(ldy=260) == MISALIGNED
    assert call(k=192) == UNSUPPORTED and call(n=252) == UNSUPPORTED
    assert call(m=(1 << 22) + 1) == UNSUPPORTED
    assert call(n=8, ldy=8) == NO_DEVICE and call() == NO_DEVICE


def test_norm_rejects_bad_arguments():
    lib = _lib.load()
    p, z = ctypes.c_void_p(FAKE), ctypes.c_void_p
    base = dict(x=p, m=4, k=256, ldx=256, r=None, ldr=0, w=p, wt=0, eps=1e-6, h=None, ldh=0, c=p, sf=p)
    for fn in (lib.svdq_rmsnorm_mxfp8, lib.svdq_rmsnorm_mxfp4):
        def call(**kw):
            a = dict(base, **kw)
            return fn(a["x"], a["m"], a["k"], a["ldx"], a["r"], a["ldr"], a["w"], a["wt"], a["eps"], a["h"], a["ldh"],
                      a["c"], a["sf"], None)

        both = dict(r=p, ldr=256, h=p, ldh=256)
        for name in ("x", "w", "c", "sf"):
            assert call(**{name: None}) == INVALID
            assert call(**{name: z(FAKE + 2)}) == MISALIGNED
        assert call(r=p, ldr=256) == INVALID                                # a residual without H
        assert call(h=p, ldh=256) == INVALID                                # H without a residual
        assert call(m=0) == INVALID and call(k=0) == INVALID and call(ldx=128) == INVALID
        assert call(**dict(both, ldr=128)) == INVALID and call(**dict(both, ldh=248)) == INVALID
        assert call(**dict(both, ldr=260)) == MISALIGNED and call(**dict(both, ldh=260)) == MISALIGNED
        assert call(**dict(both, h=z(FAKE + 8))) == MISALIGNED
        assert call(wt=2) == INVALID
        for eps in (0.0, -1e-6, float("nan"), float("inf")):
            assert call(eps=eps) == INVALID
        assert call(k=320, ldx=320) == UNSUPPORTED
        assert call(k=(1 << 30) + 128, ldx=(1 << 30) + 128) == UNSUPPORTED
        assert call() == NO_DEVICE and call(**both) == NO_DEVICE and call(wt=1) == NO_DEVICE


def test_debug_sites():
    from bit_w4a4_quantized_svdq_b200.build import DEBUG_LIB_PATH
    dbg = ctypes.CDLL(DEBUG_LIB_PATH)
    dbg.svdq_debug_limit_extent.argtypes = [ctypes.c_int, ctypes.c_int64]
    for site in (32, 33, 34):
        assert dbg.svdq_debug_limit_extent(site, 0) == 0
    for site in (17, 31, 35, 1000):
        assert dbg.svdq_debug_limit_extent(site, 0) == INVALID


# ------------------------------------------------------------------------------------------ the binding
class _Recorder:
    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name.endswith("_sf_bytes") or name == "svdq_status_string":
            return getattr(self.real, name)

        def call(*args):
            self.calls.append((name, args))
            return _lib.SVDQ_OK
        return call


@pytest.fixture
def rec(monkeypatch):
    r = _Recorder(_lib.load())
    monkeypatch.setattr(_lib, "load", lambda path=None: r)
    monkeypatch.setattr(_lib, "out_empty", lambda shape, dtype, device: torch.empty(shape, dtype=dtype))
    monkeypatch.setattr(ops, "_stream", lambda stream: None)

    def check_bf16_host(t, name):            # the dtype part of the check; the device part needs a GPU
        if t.dtype not in ops._BF16_TYPES:
            raise TypeError(name)
    monkeypatch.setattr(ops, "_check_bf16", check_bf16_host)
    return r


def _bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_quantize_and_dequantize_marshalling(rec):
    wide = _bf16(5, 300)
    q = ops.svdq_quantize_mxfp4.__wrapped__(wide[:, :256])
    assert q["codes"].shape == (5, 128) and q["sf"].numel() == 128 * 8
    assert rec.calls[-1] == ("svdq_quantize_mxfp4", (wide.data_ptr(), 5, 256, 300, q["codes"].data_ptr(),
                                                     q["sf"].data_ptr(), None))
    y = ops.svdq_dequantize_mxfp4.__wrapped__(q["codes"], q["sf"])
    assert y.shape == (5, 256) and rec.calls[-1][1] == (q["codes"].data_ptr(), q["sf"].data_ptr(), 5, 256, y.data_ptr(), 256, None)
    out = _bf16(5, 200)[:, :128]
    ops.svdq_dequantize_mxfp8.__wrapped__(q["codes"], torch.zeros(128 * 4, dtype=torch.uint8), out=out)
    assert rec.calls[-1][0] == "svdq_dequantize_mxfp8" and rec.calls[-1][1][2:] == (5, 128, out.data_ptr(), 200, None)
    n = len(rec.calls)
    for bad, err in ((lambda: ops.svdq_quantize_mxfp4.__wrapped__(_bf16(5, 192)), ValueError),
                     (lambda: ops.svdq_quantize_mxfp4.__wrapped__(_bf16(0, 128)), ValueError),
                     (lambda: ops.svdq_quantize_mxfp4.__wrapped__(torch.zeros(5, 128)), TypeError),
                     (lambda: ops.svdq_quantize_mxfp4.__wrapped__(_bf16(128, 8).t()), ValueError),
                     (lambda: ops.svdq_quantize_mxfp4.__wrapped__(wide[:, :256], out=dict(q, sf=q["sf"][:-1])), ValueError),
                     (lambda: ops.svdq_dequantize_mxfp4.__wrapped__(q["codes"], q["sf"][:-1]), ValueError),
                     (lambda: ops.svdq_dequantize_mxfp4.__wrapped__(q["codes"].to(torch.int8), q["sf"]), TypeError),
                     (lambda: ops.svdq_dequantize_mxfp4.__wrapped__(q["codes"], q["sf"], out=_bf16(5, 128)), ValueError),
                     (lambda: ops.svdq_dequantize_mxfp4.__wrapped__(q["codes"].view(-1), q["sf"]), ValueError)):
        with pytest.raises(err):
            bad()
    assert len(rec.calls) == n


def test_linear_marshalling(rec):
    ac, wc = torch.zeros((3, 64), dtype=torch.uint8), torch.zeros((136, 64), dtype=torch.uint8)
    asf, wsf = torch.zeros(512, dtype=torch.uint8), torch.zeros(1024, dtype=torch.uint8)
    y = ops.svdq_linear_mxfp4.__wrapped__(ac, asf, wc, wsf)
    assert rec.calls[-1] == ("svdq_linear_mxfp4", (ac.data_ptr(), asf.data_ptr(), wc.data_ptr(), wsf.data_ptr(), None,
                                                   y.data_ptr(), 136, 3, 136, 128, None))
    n = len(rec.calls)
    for args, kw, err in (((ac, asf[:-1], wc, wsf), {}, ValueError), ((ac, asf, wc, asf), {}, ValueError),
                          ((ac, asf, wc[:, :32], wsf), {}, ValueError), ((ac.to(torch.int8), asf, wc, wsf), {}, TypeError),
                          ((ac, asf, wc, wsf, _bf16(135)), {}, ValueError), ((ac, asf, wc, wsf, torch.zeros(136)), {}, TypeError),
                          ((ac, asf, wc, wsf), dict(out=_bf16(3, 128)), ValueError),
                          ((ac, asf, wc, wsf), dict(out=torch.zeros(3, 136)), ValueError),
                          ((ac, asf, wc, wsf), dict(out=_bf16(136, 3).t()), ValueError)):
        with pytest.raises(err):
            ops.svdq_linear_mxfp4.__wrapped__(*args, **kw)
    assert len(rec.calls) == n


@pytest.mark.parametrize("name,per_byte", [("svdq_rmsnorm_mxfp8", 1), ("svdq_rmsnorm_mxfp4", 2)])
def test_norm_marshalling(rec, name, per_byte):
    fn = getattr(ops, name).__wrapped__
    x, r, w = _bf16(3, 300)[:, :256], _bf16(3, 256), torch.zeros(256)
    q = fn(x, w, eps=1e-5)
    got = rec.calls[-1]
    assert got[0] == name and q["h"] is None and q["codes"].shape == (3, 256 // per_byte)
    assert got[1] == (x.data_ptr(), 3, 256, 300, None, 0, w.data_ptr(), 1, 1e-5, None, 0, q["codes"].data_ptr(),
                      q["sf"].data_ptr(), None)
    q = fn(x, w.to(torch.bfloat16), r, out=dict(q, h=r))
    got = rec.calls[-1][1]
    assert got[4:6] == (r.data_ptr(), 256) and got[7] == 0 and got[9:11] == (r.data_ptr(), 256) and q["h"] is r
    q = fn(x, w, r, out=dict(codes=q["codes"], sf=q["sf"]))                 # h made by the call
    assert q["h"].shape == (3, 256) and rec.calls[-1][1][9] == q["h"].data_ptr()
    n = len(rec.calls)
    for args, kw, err in (((x, w[:-1]), {}, ValueError), ((x, w.double()), {}, TypeError), ((x, w, r[:2]), {}, ValueError),
                          ((x, w, r.float()), {}, TypeError), ((x.float(), w), {}, TypeError),
                          ((x, w), dict(out=q), ValueError),                # h without a residual
                          ((x, w, r), dict(out=dict(q, h=r[:2])), ValueError),
                          ((x, w, r), dict(out=dict(q, h=r.float())), ValueError),
                          ((x, w, r), dict(out=dict(q, codes=q["codes"][:2])), ValueError),
                          ((x, torch.zeros(512)[::2]), {}, ValueError)):
        with pytest.raises(err):
            fn(*args, **kw)
    assert len(rec.calls) == n


def test_calls_refuse_cpu_tensors():
    with pytest.raises(ValueError, match="CUDA tensors"):
        ops.svdq_quantize_mxfp4(_bf16(4, 128))
    with pytest.raises(ValueError, match="CUDA tensors"):
        ops.svdq_rmsnorm_mxfp8(_bf16(4, 128), torch.ones(128))
