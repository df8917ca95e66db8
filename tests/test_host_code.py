"""Host code of the library that no call reaches without a device or a failure:
small programs compiled against its sources, which play the CUDA runtime's part
themselves (no device is touched)."""
import os
import subprocess

from weight_gradient_gemm_gb300 import _build


def run(tmp_path, program, runtime, objects=()):
    """Compiles `program` (CUDA C++) with `runtime` (C++: the runtime's functions it
    replaces) and the objects given, and runs it."""
    paths = [os.path.join(tmp_path, n) for n in ("program.cu", "runtime.cpp", "program")]
    for path, text in zip(paths, (program, runtime)):
        with open(path, "w") as f:
            f.write(text)
    lib = os.path.join(os.path.dirname(os.path.dirname(_build.nvcc())), "lib64")
    cmd = ([_build.nvcc()] + _build.ARCH + ["-O1", "-std=c++17", "--expt-relaxed-constexpr",
           "-I", os.path.join(_build.ROOT, "include"), "-I", _build.CSRC, "-cudart", "shared",
           "-Xlinker", "-rpath," + lib, "-o", paths[2]] + paths[:2] + list(objects))
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([paths[2]], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_a_failed_launch_leaves_no_error_behind(tmp_path):
    # the check after another launch must not meet the error
    run(tmp_path, """
#include <cstdio>
#include "forge_launch.cuh"
extern cudaError_t last_error;
__global__ void nothing(int) {}
int main() {
  const cudaError_t e = forge::launch_chained(nothing, 1, 32, 0, 0, nullptr, 1);
  std::printf("%d, left %d\\n", static_cast<int>(e), static_cast<int>(last_error));
  return e == cudaErrorInvalidConfiguration && last_error == cudaSuccess ? 0 : 1;
}
""", """
#include <cuda_runtime_api.h>
cudaError_t last_error = cudaSuccess;
extern "C" cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t*, const void*, void**) {
  return last_error = cudaErrorInvalidConfiguration;
}
extern "C" cudaError_t cudaGetLastError() {
  const cudaError_t e = last_error;
  last_error = cudaSuccess;
  return e;
}
""")
