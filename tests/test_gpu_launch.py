"""Host helpers that the kernels' launches share (without a driver every call reports an error)."""
import os
import subprocess

import pytest

from paged_kv_chunk_query_b200 import build

pytestmark = pytest.mark.gpu

PROGRAM = r"""
#include "launch.cuh"
int main() {
  cudaGetLastError();
  if (oomb::sm_count(12345) != 148) return 1;             // no such device
  return cudaGetLastError() == cudaSuccess ? 0 : 2;       // what the next launch would report
}
"""


def test_an_unknown_device_leaves_no_error_for_the_next_launch(tmp_path):
    if not os.path.exists(build.NVCC):
        pytest.skip("no nvcc")
    src, exe = tmp_path / "t.cu", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run([build.NVCC, *build.ARCH, "-std=c++17", "-I", build.CSRC, "-o", exe, src],
                   check=True, capture_output=True, text=True)
    assert subprocess.run([exe], timeout=120).returncode == 0
