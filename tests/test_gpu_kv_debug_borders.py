"""The KV cache's border cases on the bounds-checking build, in a process of their own (tests/conftest.py reads the status
after each test)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_kv_cache_borders_on_the_bounds_checking_build():
    lib = os.path.join(ROOT, "qad_nvfp4_quantize_b200", "libnvfp4_debug.so")
    if not os.path.exists(lib):
        pytest.fail(f"{lib} is missing; build it with `python -m qad_nvfp4_quantize_b200.build --debug`")
    res = subprocess.run([sys.executable, "-m", "pytest", "tests/test_gpu_kv_cache_borders.py", "-m", "gpu", "-q", "-x", "-p",
                          "no:cacheprovider"],
                         cwd=ROOT, env=dict(os.environ, NVFP4_LIBRARY="debug"), capture_output=True, text=True, timeout=900)
    tail = "\n".join((res.stdout + res.stderr).strip().splitlines()[-25:])
    assert res.returncode == 0 and " passed" in res.stdout, tail
