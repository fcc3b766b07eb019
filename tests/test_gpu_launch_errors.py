"""GPU test of the launch helpers (csrc/kvarn_block_dev.cuh): an error that a call has returned does not stay behind, where the
next call would take it for its own. A launch of no thread blocks and more shared memory than there is are refused by the runtime
before anything reaches the GPU."""
import subprocess

import pytest

from quantized_kv_cache_seal_gb300 import build

pytestmark = pytest.mark.gpu

PROGRAM = r"""
#include <cstdio>
#include "kvarn_block_dev.cuh"
__global__ void nothing(int) {}
int main() {
    const int launch = kvarn::launch_behind(nothing, dim3(0), 32, 0, nullptr, 0);
    const int after = (int)cudaGetLastError();
    kvarn::SmemOnce once;
    const int allow = once.allow(reinterpret_cast<const void*>(nothing), 1 << 30);
    std::printf("%d %d %d %d\n", launch, after, allow, (int)cudaGetLastError());
}
"""


def test_errors_belong_to_the_call_that_made_them(tmp_path):
    source, program = tmp_path / "launch.cu", tmp_path / "launch"
    source.write_text(PROGRAM)
    subprocess.run([build._nvcc(), str(source), "-o", str(program)] + build._flags(), check=True, capture_output=True)
    out = subprocess.run([str(program)], check=True, capture_output=True, text=True).stdout
    launch, after_launch, allow, after_allow = map(int, out.split())
    assert launch != 0 and allow != 0
    assert after_launch == 0 and after_allow == 0
