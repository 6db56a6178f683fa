"""The edge and stream tests of the MXFP4 operators and the norms again, against the debug
library: a child pytest with SVDQ_DEBUG=1, as test_gpu_mx4_debug.py runs the main suite."""
import os
import re
import subprocess
import sys

import pytest

from gpu_util import requires_cuda

pytestmark = [pytest.mark.gpu, requires_cuda]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FILES = ["tests/test_gpu_mx4_edges.py", "tests/test_gpu_mx4_streams.py"]


def test_mx4_edges_and_streams_under_the_debug_library():
    env = dict(os.environ, SVDQ_DEBUG="1")
    res = subprocess.run([sys.executable, "-m", "pytest", *FILES, "-m", "gpu", "-x", "-q", "-p", "no:cacheprovider"],
                         cwd=ROOT, env=env, capture_output=True, text=True, timeout=1200)
    tail = res.stdout[-6000:] + res.stderr[-3000:]
    assert res.returncode == 0, tail
    passed = re.search(r"(\d+) passed", res.stdout)
    assert passed and int(passed.group(1)) >= 20 and "skipped" not in res.stdout.splitlines()[-1], tail
