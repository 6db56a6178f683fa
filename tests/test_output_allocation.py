"""Outputs come from torch's public allocation call: dispatch modes see each of them, any shape
is laid out contiguously, and torch's deterministic fill applies.  (On CPU nothing is allocated on a
device: the mode answers on the host.)"""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from bit_w4a4_quantized_svdq_b200 import _lib

pytestmark = pytest.mark.skipif(_lib.DEBUG, reason="debug outputs are views of guarded buffers")


class _OnTheHost(TorchDispatchMode):
    """Records each operation that names a device and runs it on the CPU."""

    def __init__(self):
        super().__init__()
        self.seen = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        kwargs = dict(kwargs or {})
        if "device" in kwargs:
            self.seen.append((str(func), list(args[0]), kwargs["device"]))
            kwargs["device"] = torch.device("cpu")
        return func(*args, **kwargs)


@pytest.mark.parametrize("shape,sizes", [((), []), (7, [7]), ((0,), [0]), ((3, 5), [3, 5]), ((2, 3, 4), [2, 3, 4])])
def test_outputs_go_through_the_dispatcher(monkeypatch, shape, sizes):
    monkeypatch.setattr(torch.cuda, "_lazy_init", lambda: None)
    dev = torch.device("cuda", 0)
    with _OnTheHost() as mode:
        t = _lib.out_empty(shape, torch.bfloat16, dev)
    assert mode.seen == [("aten.empty.memory_format", sizes, dev)]
    assert t.dtype == torch.bfloat16 and list(t.shape) == sizes and t.is_contiguous()


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA device")
def test_outputs_follow_the_deterministic_fill():
    """With torch's deterministic mode on, memory a call has not written yet reads as NaN."""
    before = torch.are_deterministic_algorithms_enabled(), torch.is_deterministic_algorithms_warn_only_enabled()
    torch.use_deterministic_algorithms(True)
    try:
        t = _lib.out_empty((3, 5), torch.bfloat16, torch.device("cuda", torch.cuda.current_device()))
    finally:
        torch.use_deterministic_algorithms(before[0], warn_only=before[1])
    assert bool(torch.isnan(t).all())
