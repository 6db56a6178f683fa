"""Calls from several host threads at once, each on a stream of its own; an exception in any thread,
or a thread that did not finish its rounds, fails the test.  Run under the debug library too, where
a call's guard bands and the device error word are checked after each call."""
import threading

import pytest
import torch

from gpu_util import requires_cuda
from test_gpu_mx4 import _block, _block_state

pytestmark = [pytest.mark.gpu, requires_cuda]

ROUNDS = 30


@pytest.fixture(scope="module")
def lib():
    import bit_w4a4_quantized_svdq_b200 as P
    return P


def _run_threads(work, items):
    """work(item) for every item in a thread each, started together; returns the failures."""
    failures, done, start = [], [], threading.Barrier(len(items))

    def body(item):
        try:
            start.wait(timeout=60)
            done.append(work(item))
        except BaseException as e:  # noqa: BLE001 -- reported below, whatever it is
            failures.append(f"{type(e).__name__}: {e}")

    threads = [threading.Thread(target=body, args=(i,)) for i in items]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=600)
    assert not any(t.is_alive() for t in threads)
    assert not failures, failures
    return done


@pytest.mark.parametrize("given", [True, False])               # the stream as an argument, or current in the thread
def test_threads_on_their_own_streams(lib, given):
    states = [_block_state(lib, m, 1280, 170 + m) for m in (2, 300, 40)]
    want = [[t.clone() for t in _block(lib, s)] for s in states]
    torch.cuda.synchronize()

    def work(item):
        s, w = item
        st = torch.cuda.Stream()
        for i in range(ROUNDS):
            if given:
                got = _block(lib, s, stream=st)
            else:
                with torch.cuda.stream(st):
                    got = _block(lib, s)
            st.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, w)):
                raise AssertionError(f"round {i} of {s['x'].shape[0]} rows differs")
        return ROUNDS

    assert _run_threads(work, list(zip(states, want))) == [ROUNDS] * len(states)
    assert lib.svdq_device_error() == 0


def test_an_exception_in_a_thread_is_seen(lib):
    """The scheme above reports a call that raises (here: columns that are not a multiple of 128)."""
    x = torch.zeros((4, 192), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(AssertionError, match="ValueError"):
        _run_threads(lambda item: lib.svdq_quantize_mxfp4(item), [x, x])
