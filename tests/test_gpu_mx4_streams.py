"""Calls given a stream, as a program that overlaps them uses them: the outputs are read on
the calling stream after it has waited for the given one, then released."""
import pytest
import torch

from gpu_util import requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]


@pytest.fixture(scope="module")
def lib():
    import bit_w4a4_quantized_svdq_b200 as P
    return P


def _x(m, k, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(m, k, device="cuda", generator=g).to(torch.bfloat16)


# The inputs `i` exist before either stream runs, so the given
# stream has nothing to wait for.
CALLS = {"quantise mxfp8": lambda lib, x, i, **kw: lib.svdq_quantize_mxfp8(x, **kw),
         "quantise mxfp4": lambda lib, x, i, **kw: lib.svdq_quantize_mxfp4(x, **kw),
         "quantise nvfp4": lambda lib, x, i, **kw: lib.svdq_quantize_act(x, None, i["one"], **kw),
         "norm": lambda lib, x, i, **kw: lib.svdq_rmsnorm_mxfp4(x, i["ones"], x, **kw),
         "read back": lambda lib, x, i, **kw: dict(y=lib.svdq_dequantize_mxfp4(x.view(torch.uint8), i["sf"], **kw)),
         "linear": lambda lib, x, i, **kw: dict(y=lib.svdq_linear_mxfp4(x.view(torch.uint8), i["sf"], i["w"]["codes"],
                                                                       i["w"]["sf"], **kw))}


@pytest.mark.parametrize("name", list(CALLS))
def test_output_released_while_the_calling_stream_still_reads_it(lib, name):
    """The memory of a released output goes to no later call before the reads that the calling
    stream had queued are done.  (The caller waits for the given stream, as it always had to.)"""
    x1, x2 = _x(1000, 1024, 1), _x(1000, 1024, 2)
    # x's bytes serve as MXFP4 codes [1000, 2048] too
    inputs = dict(ones=torch.ones(1024, device="cuda"), one=torch.ones(1, device="cuda"),
                  sf=lib.svdq_quantize_mxfp4(_x(1000, 4096, 4))["sf"], w=lib.svdq_quantize_mxfp4(_x(1024, 4096, 5)))

    def call(lib, x, **kw):
        return CALLS[name](lib, x, inputs, **kw)

    want = {k: t.clone() for k, t in call(lib, x1).items() if t is not None}
    busy = torch.zeros(1 << 28, device="cuda")
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    out = {k: t for k, t in call(lib, x1, stream=side).items() if t is not None}
    here.wait_stream(side)
    for _ in range(40):                                       # about 10 ms of work before the reads below
        busy.add_(1.0)
    got = {k: t.clone() for k, t in out.items()}
    del out
    for _ in range(3):
        call(lib, x2, stream=side)
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(got[k].view(torch.uint8), want[k].view(torch.uint8)), k
    assert lib.svdq_device_error() == 0


def test_output_of_a_call_given_the_calling_stream(lib):
    x = _x(64, 512, 3)
    want = lib.svdq_quantize_mxfp4(x)
    got = lib.svdq_quantize_mxfp4(x, stream=torch.cuda.current_stream())
    assert torch.equal(got["codes"], want["codes"]) and torch.equal(got["sf"], want["sf"])


def test_callers_buffers_keep_their_own_stream(lib):
    """Buffers passed as `out` come back as they are."""
    x, side = _x(64, 512, 4), torch.cuda.Stream()
    want = lib.svdq_quantize_mxfp4(x)
    out = {k: torch.empty_like(t) for k, t in want.items()}
    torch.cuda.synchronize()
    q = lib.svdq_quantize_mxfp4(x, out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert q["codes"] is out["codes"] and q["sf"] is out["sf"]
    assert torch.equal(q["codes"], want["codes"]) and torch.equal(q["sf"], want["sf"])


def test_captured_on_a_side_stream(lib):
    """A captured call given a joined stream: the graph replays, and its outputs stay its own."""
    x, w, side = _x(33, 640, 5), torch.ones(640, device="cuda"), torch.cuda.Stream()
    want = lib.svdq_rmsnorm_mxfp8(x, w, x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        dropped = lib.svdq_quantize_mxfp4(x, stream=side)     # released during the capture
        del dropped
        out = lib.svdq_rmsnorm_mxfp8(x, w, x, stream=side)
        here.wait_stream(side)
    for _ in range(3):
        for t in out.values():
            t.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], want[k]) for k in want)
