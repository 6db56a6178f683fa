"""What is measured of the microscaled operators: RMS norm into MXFP8 and MXFP4, the MXFP4 quantiser with
its read-back, the MXFP4 linear, and the norm followed by the linear.

``run`` computes each operator in elementary torch operations (``own`` false) or by the framework's calls
(``own`` true); ``exact`` computes the definition in 64 bits.  Sizes follow the configured layers: rows of
one token, of the packed text rows (29, 115), and of whole packed sequences (4096, 16384); channels 5120 and
20480; fused and plain projections (5120, 15360 columns).

Storage formats (as the library documents them): E4M3 codes one byte an element; E2M1 codes two a byte,
element 2i in the low nibble; one E8M0 scale byte per 32 consecutive elements, in 512-byte atoms of 128 rows
by 4 blocks, row r's four bytes at (r % 32) * 16 + (r / 32 % 4) * 4, atoms along the row first.
"""
import math

import torch

own = False

EPS = 1e-6

# Largest magnitude's exponent and mantissa bits of each element format.
FORMATS = {"mxfp8": dict(emax=8, emin=-6, mant=3, top=448.0), "mxfp4": dict(emax=2, emin=0, mant=1, top=6.0)}


# ---------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # one token entering a block: the norm's latency
        dict(name="norm8 one token", op="norm", fmt="mxfp8", m=1, k=5120, res=True, w32=False),
        # a first norm without a residual, ragged rows, a narrow width that is no power of two, fp32 weight
        dict(name="norm8 ragged", op="norm", fmt="mxfp8", m=1037, k=1920, res=False, w32=True),
        # every norm of a block over a whole packed sequence
        dict(name="norm8 sequence", op="norm", fmt="mxfp8", m=16384, k=5120, res=True, w32=False),
        # the text rows of a packed sequence, quantised and read back
        dict(name="quant4 text rows", op="quant", m=115, k=5120),
        # the FFN down-projection's input
        dict(name="quant4 FFN", op="quant", m=16384, k=20480),
        # one token through a projection: the weight is what has to be read
        dict(name="linear4 one token", op="linear", m=1, n=5120, k=5120, bias=True),
        # text rows through the fused query, key and value projection
        dict(name="linear4 text rows", op="linear", m=29, n=15360, k=5120, bias=True),
        # ragged rows and columns, no bias
        dict(name="linear4 ragged", op="linear", m=515, n=1160, k=1920, bias=False),
        # attention projection of a packed sequence
        dict(name="linear4 attention", op="linear", m=4096, n=5120, k=5120, bias=True),
        # FFN down-projection of the longest packed sequence
        dict(name="linear4 FFN down", op="linear", m=16384, n=5120, k=20480, bias=True),
        # norm with residual, 4-bit output, and the projection that reads it: one token, a whole sequence
        dict(name="block4 one token", op="block", m=1, n=5120, k=5120, bias=True),
        dict(name="block4 sequence", op="block", m=4096, n=15360, k=5120, bias=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the same ranges: rows 1..16384, channels a multiple of 128 up to 20480 (a norm's: 8192),
    columns a multiple of 8 up to 20480; none costs more than the largest listed one."""
    op = rng.choice(["norm", "norm", "quant", "linear", "linear", "linear", "block"])
    m = _log_int(rng, 1, 16384)
    if op == "norm":
        return dict(op="norm", fmt=rng.choice(["mxfp8", "mxfp8", "mxfp4"]), m=m, k=128 * _log_int(rng, 1, 64),
                    res=rng.random() < 0.7, w32=rng.random() < 0.4)
    if op == "quant":
        return dict(op="quant", m=m, k=128 * _log_int(rng, 1, 160))
    n = 8 * _log_int(rng, 16, 2560)
    k = 128 * _log_int(rng, 1, 160 if op == "linear" else 64)
    while m * n * k > 16384 * 5120 * 20480:
        m = max(1, m // 2)
    return dict(op=op, m=m, n=n, k=k, bias=rng.random() < 0.6)


def work(case):
    m, k = case["m"], case["k"]
    code_bytes = {"mxfp8": 1.0, "mxfp4": 0.5}
    per_row = lambda fmt: k * code_bytes[fmt] + k / 32      # codes and scale bytes of one row  # noqa: E731
    if case["op"] == "norm":
        b = m * 2 * k * (3 if case["res"] else 1) + k * (4 if case["w32"] else 2) + m * per_row(case["fmt"])
        return {"bytes": b, "flops": 6.0 * m * k}
    if case["op"] == "quant":                               # quantise, then read back: codes written and read
        return {"bytes": m * (2 * k + 2 * per_row("mxfp4") + 2 * k), "flops": 4.0 * m * k}
    n = case["n"]
    b = n * per_row("mxfp4") + 2.0 * m * n + (2 * n if case["bias"] else 0)
    if case["op"] == "linear":
        b += m * per_row("mxfp4")
    else:                                                   # x, residual, their sum; the codes between the two calls
        b += m * 6 * k + 2 * k + 2 * m * per_row("mxfp4")
    return {"bytes": b, "flops": 2.0 * m * n * k}


# ----------------------------------------------------------------------------------- plain element formats
def _pow2(e):
    """2^e in fp32 for whole e in [-127, 127]."""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).to(torch.int32).view(torch.float32)


def _exponent(v):
    """Biased fp32 exponent field of v (0 for zero and subnormals)."""
    return (v.view(torch.int32) >> 23) & 0xFF


def _round_to(v, fmt):
    """fp32 -> nearest value of the element format, ties to even, saturating, sign kept."""
    f = FORMATS[fmt]
    a = v.abs()
    e = (_exponent(a) - 127).clamp_(f["emin"], f["emax"])
    a = torch.round(a * _pow2(f["mant"] - e)) * _pow2(e - f["mant"])
    return torch.copysign(a.clamp_(max=f["top"]), v)


def _mx_quantise(v, fmt):
    """fp32 [M, K] -> element values (fp32) and scale exponents (int32 [M, K / 32])."""
    m, k = v.shape
    b = v.reshape(m, k // 32, 32)
    field = _exponent(b.abs().amax(-1))
    e = torch.where(field == 0, torch.full_like(field, -127), (field - 127 - FORMATS[fmt]["emax"]).clamp(min=-127))
    return _round_to(b * _pow2(-e).unsqueeze(-1), fmt).reshape(m, k), e


def _tile_scales(e):
    """Scale exponents [rows, blocks] -> bytes in atoms, rows padded to 128 with zero bytes."""
    rows, blocks = e.shape
    pad = -rows % 128
    b = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, 0, 0, pad))
    return b.view((rows + pad) // 128, 4, 32, blocks // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _untile_scales(sf, rows, blocks):
    """Bytes in atoms -> scale exponents int32 [rows, blocks]."""
    b = sf.view(-1, blocks // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, blocks)[:rows]
    return b.to(torch.int32) - 127


def _pack4(v):
    """Element values of MXFP4 -> packed nibbles."""
    a = v.abs()
    mag = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    c = mag | (torch.signbit(v).to(torch.uint8) << 3)
    return c[:, 0::2] | (c[:, 1::2] << 4)


def _unpack4(codes):
    """Packed nibbles -> fp32 element values."""
    m, kh = codes.shape
    c = torch.stack((codes & 15, codes >> 4), dim=-1).view(m, 2 * kh)
    mag = (c & 7).to(torch.float32)
    a = torch.where(mag < 4, mag * 0.5, torch.where(mag < 6, mag - 2, mag * 2 - 8))
    return torch.where(c > 7, -a, a)


def _values4(codes, sf):
    m, k = codes.shape[0], 2 * codes.shape[1]
    v = _unpack4(codes).view(m, k // 32, 32)
    return v.mul_(_pow2(_untile_scales(sf, m, k // 32)).unsqueeze(-1)).view(m, k)


# --------------------------------------------------------------------------------------------- the inputs
def _activations(m, k, g):
    """Channel profiles with a few large channels, as the activations of a block have them."""
    p = torch.exp(0.75 * torch.randn(k, generator=g, device="cuda"))
    big = torch.rand(k, generator=g, device="cuda") < 0.01
    p = torch.where(big, p * (20 + 80 * torch.rand(k, generator=g, device="cuda")), p)
    return (torch.randn(m, k, generator=g, device="cuda") * p).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + 17)
    m, k, op = case["m"], case["k"], case["op"]
    s = dict(case=dict(case))
    x = _activations(m, k, g)
    if op == "linear":                                      # the activations arrive quantised
        v, e = _mx_quantise(x.float(), "mxfp4")
        s["a_codes"], s["a_sf"] = _pack4(v), _tile_scales(e)
    else:
        s["x"] = x
    if op in ("norm", "block"):
        w = 1.0 + 0.2 * torch.randn(k, generator=g, device="cuda")
        s["weight"] = w if case.get("w32") else w.to(torch.bfloat16)
        s["residual"] = _activations(m, k, g) if case.get("res", True) else None
    if op in ("linear", "block"):                           # a converted weight and its bias
        n = case["n"]
        v, e = _mx_quantise((0.02 * torch.randn(n, k, generator=g, device="cuda")).to(torch.bfloat16).float(), "mxfp4")
        s["w_codes"], s["w_sf"] = _pack4(v), _tile_scales(e)
        s["bias"] = (0.02 * torch.randn(n, generator=g, device="cuda")).to(torch.bfloat16) if case["bias"] else None
    return s


# ---------------------------------------------------------------------------------------------- one pass
def _plain_norm(s):
    """h (bf16, or None without a residual) and the normalised rows in fp32; the sum of squares in 64 bits."""
    h = s["x"]
    if s["residual"] is not None:
        h = (h.float() + s["residual"].float()).to(torch.bfloat16)
    v = h.float()
    mean = v.double().square().mean(-1, keepdim=True)
    rstd = torch.rsqrt(mean + EPS).float()
    return (h if s["residual"] is not None else None), (v * rstd) * s["weight"].float()


def _plain_linear(a, s):
    y = a @ _values4(s["w_codes"], s["w_sf"]).t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(torch.bfloat16)


def _outputs(h, **more):
    return more if h is None else dict(h=h, **more)


def run(state):
    s = state
    op, fmt = s["case"]["op"], s["case"].get("fmt")
    if own:
        import bit_w4a4_quantized_svdq_b200 as P
        if op == "norm":
            norm = P.svdq_rmsnorm_mxfp8 if fmt == "mxfp8" else P.svdq_rmsnorm_mxfp4
            q = norm(s["x"], s["weight"], s["residual"], eps=EPS)
            if fmt == "mxfp8":                              # 8 bits a value: the bytes under their own types
                return _outputs(q["h"], codes=q["codes"].view(torch.float8_e4m3fn), sf=q["sf"].view(torch.float8_e8m0fnu))
            return _outputs(q["h"], values=P.svdq_dequantize_mxfp4(q["codes"], q["sf"]))
        if op == "quant":
            q = P.svdq_quantize_mxfp4(s["x"])
            return P.svdq_dequantize_mxfp4(q["codes"], q["sf"])
        if op == "linear":
            return P.svdq_linear_mxfp4(s["a_codes"], s["a_sf"], s["w_codes"], s["w_sf"], s["bias"])
        q = P.svdq_rmsnorm_mxfp4(s["x"], s["weight"], s["residual"], eps=EPS)
        y = P.svdq_linear_mxfp4(q["codes"], q["sf"], s["w_codes"], s["w_sf"], s["bias"])
        return _outputs(q["h"], y=y)
    if op == "norm":
        h, y = _plain_norm(s)
        v, e = _mx_quantise(y, fmt)
        if fmt == "mxfp8":
            return _outputs(h, codes=v.to(torch.float8_e4m3fn), sf=_tile_scales(e).view(torch.float8_e8m0fnu))
        return _outputs(h, values=(v.view(e.shape + (32,)) * _pow2(e).unsqueeze(-1)).view(v.shape).to(torch.bfloat16))
    if op == "quant":
        v, e = _mx_quantise(s["x"].float(), "mxfp4")
        return (v.view(e.shape + (32,)) * _pow2(e).unsqueeze(-1)).view(v.shape).to(torch.bfloat16)
    if op == "linear":
        return _plain_linear(_values4(s["a_codes"], s["a_sf"]), s)
    h, y = _plain_norm(s)
    v, e = _mx_quantise(y, "mxfp4")
    a = (v.view(e.shape + (32,)) * _pow2(e).unsqueeze(-1)).view(v.shape)
    return _outputs(h, y=_plain_linear(a, s))


# ------------------------------------------------------------------------------- the definition in 64 bits
def _exact_mx(v, fmt):
    """fp64 [M, K] -> element values and scale exponents in fp64, by frexp and division."""
    f = FORMATS[fmt]
    b = v.view(v.shape[0], -1, 32)
    top = b.abs().max(dim=-1).values
    e = torch.where(top > 0, (torch.frexp(top).exponent - 1 - f["emax"]).double(), torch.full_like(top, -127.0))
    e = e.clamp(-127, 127)
    q = b / torch.exp2(e).unsqueeze(-1)
    step = torch.exp2((torch.frexp(q.abs()).exponent.double() - 1).clamp(f["emin"], f["emax"]) - f["mant"])
    q = (q / step).round().mul(step).clamp(-f["top"], f["top"])
    return q, e


def _exact_table(codes):
    """Packed nibbles -> fp64 values by table."""
    t = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=codes.device)
    out = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
    out[:, 0::2] = t[(codes % 16).long()]
    out[:, 1::2] = t[(codes // 16).long()]
    return out


def _exact_offsets(rows, blocks, device):
    """Byte offset of every scale [row, block]."""
    r, b = torch.arange(rows, device=device).unsqueeze(1), torch.arange(blocks, device=device).unsqueeze(0)
    return (r // 128 * (blocks // 4) + b // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + b % 4


def _exact_read(codes, sf):
    v = _exact_table(codes)
    m, k = v.shape
    scale = torch.exp2(sf[_exact_offsets(m, k // 32, sf.device)].double() - 127)
    return v * scale.repeat_interleave(32, dim=1)


def _exact_scale_bytes(e):
    """fp64 exponents [rows, blocks] -> the values of the scale bytes in storage order (padding: 2^-127)."""
    rows, blocks = e.shape
    out = torch.full(((rows + 127) // 128 * 128 * blocks,), 2.0 ** -127, dtype=torch.float64, device=e.device)
    out[_exact_offsets(rows, blocks, e.device)] = torch.exp2(e)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op, fmt = case["op"], case.get("fmt", "mxfp4")
    if op == "linear":
        a, h = _exact_read(s["a_codes"], s["a_sf"]), None
    else:
        v, h = s["x"].double(), None
        if s.get("residual") is not None:
            h = (v + s["residual"].double()).float().to(torch.bfloat16).double()      # the stored sum is bf16
            v = h
        if op != "quant":
            v = v / torch.sqrt(v.pow(2).sum(-1, keepdim=True) / v.shape[1] + EPS) * s["weight"].double()
        q, e = _exact_mx(v, fmt)
        if op == "norm" and fmt == "mxfp8":
            return _outputs(h, codes=q.view(v.shape), sf=_exact_scale_bytes(e))
        a = (q * torch.exp2(e).unsqueeze(-1)).view(v.shape)
        if op == "norm":
            return _outputs(h, values=a)
        if op == "quant":
            return a
    y = a @ _exact_read(s["w_codes"], s["w_sf"]).t()
    if s["bias"] is not None:
        y = y + s["bias"].double()
    return y if op == "linear" else _outputs(h, y=y)
