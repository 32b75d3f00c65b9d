"""CPU: a launch that the runtime refuses is reported by its own call and leaves nothing behind for the next
one. The launch helper of the sink, rotary and cache kernels is compiled against a fake runtime whose first
launch fails."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include <cuda_runtime.h>

// The parts of the CUDA runtime that a launch touches: the last error stays until it is read.
static cudaError_t last = cudaSuccess;
static int launches = 0;
template <typename... A>
static cudaError_t fake_launch(const A&...) {
  const cudaError_t e = launches++ == 0 ? cudaErrorLaunchOutOfResources : cudaSuccess;
  if (e != cudaSuccess) last = e;
  return e;
}
static cudaError_t fake_last_error() {
  const cudaError_t e = last;
  last = cudaSuccess;
  return e;
}
#define cudaLaunchKernelEx fake_launch
#define cudaGetLastError fake_last_error
#include "internal.h"

static void kernel(int) {}

int main() {
  cudaError_t got[2];
  for (cudaError_t& e : got) e = da2::launch_chained(kernel, dim3(1), dim3(32), 0, 0, nullptr, 1);
  std::printf("%d %d %d\n", got[0] == cudaErrorLaunchOutOfResources, got[1] == cudaSuccess, last == cudaSuccess);
  // an error that was there before belongs to someone else
  last = cudaErrorInvalidValue;
  std::printf("%d %d\n", da2::launch_chained(kernel, dim3(1), dim3(32), 0, 0, nullptr, 1) == cudaSuccess,
              last == cudaErrorInvalidValue);
}
"""


def test_a_refused_launch_leaves_no_error_behind(tmp_path):
    from differential_attention_v2_b200.build import nvcc

    src, exe = tmp_path / "launch.cu", tmp_path / "launch"
    src.write_text(PROGRAM)
    subprocess.run([nvcc(), "-std=c++17", "-arch=sm_100a", "-I", os.path.join(ROOT, "include"), "-I",
                    os.path.join(ROOT, "differential_attention_v2_b200", "csrc"), "-o", str(exe), str(src)],
                   check=True, capture_output=True, text=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()
    assert out == ["1"] * 5, out
