"""The router's reciprocal against the correctly rounded one, for every float of its range."""
import ctypes
import os
import re
import subprocess

import pytest

from combine_mp_layout_gb300 import _build

pytestmark = pytest.mark.gpu

PROGRAM = r"""
#include <cstdint>
#include <cuda_runtime.h>
%s
__global__ void compare(uint32_t first, uint32_t last, unsigned long long* differ) {
  unsigned long long n = 0;
  for (uint64_t u = first + blockIdx.x * uint64_t(blockDim.x) + threadIdx.x; u < last;
       u += gridDim.x * uint64_t(blockDim.x)) {
    const float y = __uint_as_float(uint32_t(u));
    n += __float_as_uint(rcp_mid(y)) != __float_as_uint(__frcp_rn(y));
  }
  if (n) atomicAdd(differ, n);
}
extern "C" long long differing(uint32_t first, uint32_t last) {
  unsigned long long *d = nullptr, n = ~0ull;
  if (cudaMalloc(&d, 8) != cudaSuccess) return -1;
  cudaMemset(d, 0, 8);
  compare<<<1216, 256>>>(first, last, d);
  const bool ok = cudaMemcpy(&n, d, 8, cudaMemcpyDeviceToHost) == cudaSuccess;
  cudaFree(d);
  return ok ? (long long)(n) : -1;
}
"""


def test_reciprocal_is_correctly_rounded_for_every_float_of_its_range(tmp_path):
    """1 <= y < 2^126, with the function as it stands in the router's source."""
    with open(os.path.join(_build.CSRC, "mp_route.cu")) as f:
        function = re.search(r"__device__ __forceinline__ float rcp_mid\(.*?\n\}", f.read(),
                             re.S).group(0)
    src, lib = tmp_path / "rcp.cu", tmp_path / "rcp.so"
    src.write_text(PROGRAM % function)
    subprocess.run([_build.nvcc(), *_build.ARCH, "-O3", "-shared", "-Xcompiler", "-fPIC", str(src),
                    "-o", str(lib)], check=True, capture_output=True, text=True)
    differing = ctypes.CDLL(str(lib)).differing
    differing.restype = ctypes.c_longlong
    differing.argtypes = [ctypes.c_uint32] * 2
    assert differing(0x3F800000, 0x7E800000) == 0
