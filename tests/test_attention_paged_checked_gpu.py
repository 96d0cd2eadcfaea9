"""The target-side attention operators under the bounds-checked build (see test_checked_gpu.py):
the pool rows that they read and write are checked, and every test asserts a clean error word."""

import os
import subprocess
import sys

import pytest

from block_diffusion_speculative_gemm_b200 import build as Bld

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_attention_paged_under_the_bounds_checked_build():
    env = dict(os.environ, DFLASH_LIB=Bld.build(checked=True))
    sel = ("tests/test_attention_paged_paths_gpu.py::test_append_many_rows "
           "tests/test_attention_paged_paths_gpu.py::test_items_of_one_and_two_query_tiles "
           "tests/test_attention_paged_paths_gpu.py::test_many_requests "
           "tests/test_attention_paged_gpu.py::test_kv_append_paged "
           "tests/test_attention_paged_gpu.py::test_attention_paged").split()
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "-m", "gpu",
                        *sel], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
