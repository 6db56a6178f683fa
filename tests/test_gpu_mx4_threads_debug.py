"""The host-thread tests again, against the debug library: a child pytest with SVDQ_DEBUG=1."""
import os
import re
import subprocess
import sys

import pytest

from gpu_util import requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_mx4_threads_under_the_debug_library():
    env = dict(os.environ, SVDQ_DEBUG="1")
    res = subprocess.run([sys.executable, "-m", "pytest", "tests/test_gpu_mx4_threads.py", "-m", "gpu", "-x", "-q",
                          "-p", "no:cacheprovider"], cwd=ROOT, env=env, capture_output=True, text=True, timeout=900)
    tail = res.stdout[-6000:] + res.stderr[-3000:]
    assert res.returncode == 0, tail
    passed = re.search(r"(\d+) passed", res.stdout)
    assert passed and int(passed.group(1)) == 3, tail
