"""The layer's quantiser and linear right behind a kernel that lets them start early (the MX read-back),
and that writes what they read: the tensor scale, the low-rank factor, the bias.  Short calls back to
back in one set of buffers, each step's results kept and compared with one kernel at a time."""
import pytest
import torch

from gpu_util import requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]

STEPS, VARIANTS, RANK = 120, 8, 32


@pytest.fixture(scope="module")
def lib():
    import bit_w4a4_quantized_svdq_b200 as P
    return P


def _randn(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, device="cuda", generator=g).to(torch.bfloat16)


def _coded(lib, t):
    """MXFP4 codes whose read-back is a [rows, 128] tensor: what the kernel before will write."""
    return lib.svdq_quantize_mxfp4(t.view(-1, 128))


@pytest.mark.parametrize("m", [3, 200])
def test_scale_factor_and_bias_written_by_the_kernel_before(lib, m):
    k, n = 1024, 512
    x, down = _randn(1, VARIANTS, m, k), _randn(2, RANK, k)
    w = lib.svdq_quantize_act(_randn(3, n, k), None, torch.full((1,), 0.01, device="cuda"))
    s_w = torch.full((1,), 0.01, device="cuda")
    scales = torch.zeros((VARIANTS, 128), dtype=torch.bfloat16, device="cuda")
    # an fp32 of zero low half: the scales of steps 0 to 7 are 2^-8 .. 2^-1
    scales[:, 1] = torch.exp2(torch.arange(VARIANTS, device="cuda") - 8.0).to(torch.bfloat16)
    scales = [_coded(lib, s) for s in scales]
    ups = [_coded(lib, _randn(10 + i, n, RANK)) for i in range(VARIANTS)]
    biases = [_coded(lib, _randn(20 + i, n)) for i in range(VARIANTS)]
    s_buf = torch.empty((1, 128), dtype=torch.bfloat16, device="cuda")
    up_buf = torch.empty((n * RANK // 128, 128), dtype=torch.bfloat16, device="cuda")
    b_buf = torch.empty((n // 128, 128), dtype=torch.bfloat16, device="cuda")
    s_g, up, bias = s_buf.view(torch.float32)[0, :1], up_buf.view(n, RANK), b_buf.view(-1)
    s_lin = torch.ones(1, device="cuda")
    q = lib.svdq_quantize_act(x[0], None, s_w, down)

    def step(i, d, y, between=lambda: None):
        v = i % VARIANTS
        lib.svdq_dequantize_mxfp4(**scales[v], out=s_buf)
        between()
        lib.svdq_quantize_act(x[v], None, s_g, down, out=dict(codes=q["codes"], sf=q["sf"], d=d))
        between()
        lib.svdq_dequantize_mxfp4(**biases[v], out=b_buf)
        between()
        lib.svdq_dequantize_mxfp4(**ups[v], out=up_buf)
        between()
        lib.svdq_linear(q["codes"], q["sf"], s_g if i % 2 else s_lin, d, w["codes"], w["sf"], s_w, up, bias, out=y)
        between()

    total = VARIANTS + STEPS
    ds = torch.empty((total, m, RANK), device="cuda")
    ys = torch.empty((total, m, n), dtype=torch.bfloat16, device="cuda")
    for i in range(VARIANTS):                                  # one kernel at a time
        step(i, ds[i], ys[i], torch.cuda.synchronize)
    assert len({float(t.float().norm()) for t in ys[:VARIANTS]}) == VARIANTS
    for i in range(VARIANTS, total):
        step(i, ds[i], ys[i])
    torch.cuda.synchronize()
    bad = [i for i in range(VARIANTS, total) if not (torch.equal(ds[i], ds[i % VARIANTS])
                                                     and torch.equal(ys[i], ys[i % VARIANTS]))]
    assert not bad, f"steps {bad[:8]} of {STEPS} read another step's scale, factor or bias"
    assert lib.svdq_device_error() == 0
