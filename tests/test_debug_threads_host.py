"""Debug mode's checks belong to one call at a time, whichever host thread makes it (CPU: a child
process with SVDQ_DEBUG=1, whose calls only wait)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import threading, time
from bit_w4a4_quantized_svdq_b200 import _lib, ops

assert _lib.DEBUG
inside, most = 0, 0

@ops._on_tensor_device
def inner():
    global inside, most
    inside += 1
    most = max(most, inside)
    time.sleep(0.05)
    inside -= 1

@ops._on_tensor_device
def outer():
    inner()                                # a call may make another

threads = [threading.Thread(target=f) for f in (inner, outer, inner, outer)]
for t in threads:
    t.start()
for t in threads:
    t.join(timeout=60)
assert not any(t.is_alive() for t in threads)
print("most at once:", most)
"""


def test_debug_calls_run_one_at_a_time():
    res = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=dict(os.environ, SVDQ_DEBUG="1"),
                         capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr[-2000:]
    assert "most at once: 1" in res.stdout, res.stdout
