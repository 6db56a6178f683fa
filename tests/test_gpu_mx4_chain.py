"""Kernels that start while the one before still runs: short calls back to back on one
stream, every buffer written again and again, each step's results kept and compared."""
import pytest
import torch

from gpu_util import requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]

STEPS = 200


@pytest.fixture(scope="module")
def lib():
    import bit_w4a4_quantized_svdq_b200 as P
    return P


def _x(n, m, k, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(n, m, k, device="cuda", generator=g).to(torch.bfloat16)


@pytest.mark.parametrize("fmt", ["mxfp4", "mxfp8"])
@pytest.mark.parametrize("m,k", [(1, 5120), (64, 1024), (700, 5120)])
def test_codes_written_and_read_back_in_the_same_buffers(lib, fmt, m, k):
    quant, back = getattr(lib, "svdq_quantize_" + fmt), getattr(lib, "svdq_dequantize_" + fmt)
    x = _x(8, m, k, 1)
    want = []
    for t in x[:8]:                                            # one kernel at a time
        q = quant(t)
        torch.cuda.synchronize()
        want.append(back(q["codes"], q["sf"]))
        torch.cuda.synchronize()
    out, got = quant(x[0]), torch.empty((STEPS, m, k), dtype=torch.bfloat16, device="cuda")
    for i in range(STEPS):
        quant(x[i % 8], out=out)
        back(out["codes"], out["sf"], out=got[i])
    torch.cuda.synchronize()
    bad = [i for i in range(STEPS) if not torch.equal(got[i], want[i % 8])]
    assert not bad, f"steps {bad[:8]} of {STEPS} read codes of another step"


@pytest.mark.parametrize("m", [1, 40, 300])
def test_weight_sum_and_bias_written_by_the_kernel_before(lib, m):
    """The norm's weight and the linear's bias are each the output of the call before, in one buffer."""
    k, n = 1024, 512
    x, r, w = _x(8, m, k, 2), _x(8, m, k, 3), lib.svdq_quantize_mxfp4(_x(1, n, k, 5)[0])
    gains = [lib.svdq_quantize_mxfp4(t) for t in _x(8, 1, k, 4)]
    out, gain = lib.svdq_quantize_mxfp4(x[0]), torch.empty((1, k), dtype=torch.bfloat16, device="cuda")

    def step(i, h, y, between=lambda: None):
        lib.svdq_dequantize_mxfp4(**gains[i % 8], out=gain)
        between()
        q = lib.svdq_rmsnorm_mxfp4(x[i % 8], gain.view(-1), r[i % 8], out=dict(out, h=h))
        between()
        lib.svdq_dequantize_mxfp4(**gains[(i + 1) % 8], out=gain)
        between()
        lib.svdq_linear_mxfp4(q["codes"], q["sf"], w["codes"], w["sf"], gain.view(-1)[:n], out=y)
        between()

    hs = torch.empty((8 + STEPS, m, k), dtype=torch.bfloat16, device="cuda")
    ys = torch.empty((8 + STEPS, m, n), dtype=torch.bfloat16, device="cuda")
    for i in range(8):                                         # one kernel at a time
        step(i, hs[i], ys[i], torch.cuda.synchronize)
    for i in range(8, 8 + STEPS):
        step(i, hs[i], ys[i])
    torch.cuda.synchronize()
    bad = [i for i in range(8, 8 + STEPS) if not (torch.equal(hs[i], hs[i % 8]) and torch.equal(ys[i], ys[i % 8]))]
    assert not bad, f"steps {bad[:8]} of {STEPS} read another step's weight or bias"
    assert lib.svdq_device_error() == 0
