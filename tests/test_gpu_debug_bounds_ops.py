"""The HSTU_DEBUG_BOUNDS build over the 8-bit projection and the candidate
scoring against the 4-bit cache: their small-shape tests run against it in a
child process and must pass with the device status clean (each of them reads
the status word)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SELECTION = [
    "tests/test_gpu_rows.py::test_uvqk_fp8",
    "tests/test_gpu_kv4.py::test_scoring",
    "tests/test_gpu_kv4.py::test_two_graphs_share_a_workspace",
    "tests/test_gpu_kv4.py::test_one_workspace_for_calls_of_different_sizes",
]


def test_small_shapes_with_device_index_checks():
    sys.path.insert(0, ROOT)
    from pointwise_attention_b200 import build
    assert build.build(debug_bounds=True).endswith("libhstu_debug.so")
    env = dict(os.environ, HSTU_DEBUG_BOUNDS="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-p", "no:cacheprovider"] +
                       SELECTION, cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    tail = "\n".join((r.stdout + r.stderr).splitlines()[-30:])
    assert r.returncode == 0, tail
    assert " passed" in tail and "failed" not in tail, tail
