"""Host code of the library that no call reaches without a device or a failure:
small programs compiled against its sources, which play the CUDA runtime's part
themselves (no device is touched)."""
import os
import shutil
import subprocess

import pytest

from weight_gradient_gemm_gb300 import _build


def run(tmp_path, program, runtime, flags=()):
    """Compiles `program` (CUDA C++) with `runtime` (C++: the runtime's functions it
    replaces) and the flags or objects given, runs it and returns what it prints."""
    paths = [os.path.join(tmp_path, n) for n in ("program.cu", "runtime.cpp", "program")]
    for path, text in zip(paths, (program, runtime)):
        with open(path, "w") as f:
            f.write(text)
    lib = os.path.join(os.path.dirname(os.path.dirname(_build.nvcc())), "lib64")
    cmd = ([_build.nvcc()] + _build.ARCH + ["-O1", "-std=c++17", "--expt-relaxed-constexpr",
           "-I", os.path.join(_build.ROOT, "include"), "-I", _build.CSRC, "-cudart", "shared",
           "-Xlinker", "-rpath," + lib, "-o", paths[2]] + paths[:2] + list(flags))
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([paths[2]], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout


def test_a_failed_launch_leaves_no_error_behind(tmp_path):
    # the check after another launch must not meet the error
    run(tmp_path, r"""
#include <cstdio>
#include "forge_launch.cuh"
extern cudaError_t last_error;
__global__ void nothing(int) {}
int main() {
  const cudaError_t e = forge::launch_chained(nothing, 1, 32, 0, 0, nullptr, 1);
  std::printf("%d, left %d\n", static_cast<int>(e), static_cast<int>(last_error));
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


# the products' host side, with nothing behind it
API = """
#include "forge_api_ops.cu"
namespace forge {
int host_device(HostDevice*) { return 0; }
int host_drop_flag() { return 0; }
bool host_map(CUtensorMap*, const void*, CUtensorMapDataType, uint64_t, uint64_t, uint64_t,
              uint32_t, uint32_t, CUtensorMapSwizzle) { return false; }
cudaError_t launch_rmsnorm(const NormArgs&, int, cudaStream_t) { return cudaSuccess; }
int rmsnorm_bwd_blocks(int64_t, int, int) { return 0; }
cudaError_t launch_rmsnorm_bwd(const NormBwdArgs&, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_quantize_b128(const uint16_t*, uint8_t*, float*, int64_t, int64_t, int, int,
                                 const NormWait&, cudaStream_t) { return cudaSuccess; }
int grad_norm_blocks(int64_t, int) { return 0; }
cudaError_t launch_grad_norm(const GradNormArgs&, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_grad_norm_final(const double*, int, float, float*, cudaStream_t) {
  return cudaSuccess;
}
cudaError_t launch_gemm_b128(const B128Config&, bool, const B128Args&, int, cudaStream_t) {
  return cudaSuccess;
}
cudaError_t launch_gemm_b128_few(int, bool, const B128Args&, int, cudaStream_t) {
  return cudaSuccess;
}
}  // namespace forge
extern "C" void forge_get_tuning(forge_tuning*) {}
"""


def test_a_split_reduction_is_shared_evenly(tmp_path):
    # every CTA of a cluster has two blocks at least, and none two more than another
    run(tmp_path, r"""
#include <cstdio>
""" + API + r"""
int main() {
  const forge_tuning automatic = {FORGE_PROFILE_AUTO, 0, 0, 0, -1, 0, -1, -1};
  int split = 0;
  for (int sms : {148, 152, 160})
    for (int n = 16; n <= 8192; n += 112)
      for (int blocks = 1; blocks <= 400; ++blocks) {
        const B128Config c = choose_b128(1, n, blocks, automatic, sms);
        int least = blocks, most = 0;
        for (int r = 0; r < c.splits; ++r) {
          const int b = b128_first_block(r + 1, c.splits, blocks) -
                        b128_first_block(r, c.splits, blocks);
          least = b < least ? b : least;
          most = b > most ? b : most;
        }
        if (b128_first_block(0, c.splits, blocks) != 0 ||
            b128_first_block(c.splits, c.splits, blocks) != blocks || most - least > 1 ||
            (c.splits > 1 && least < 2)) {
          std::printf("%d columns, %d blocks on %d CTAs: %d to %d\n", n, blocks, c.splits, least,
                      most);
          return 1;
        }
        split += c.splits > 1;
      }
  return split > 0 ? 0 : 2;
}
""", "")


def test_product_shapes_take_their_forms(tmp_path):
    # tests/test_gpu_ops_forms.py is there for these forms; on 152 SMs
    from tests.test_gpu_ops_forms import FEW, LONG
    shapes = [(bt, k, n) for bt, k, n in LONG] + [(bt, 1040, n) for bt, n in FEW]
    out = run(tmp_path, '#include <cstdio>\n' + API + r"""
int main() {
  const forge_tuning automatic = {FORGE_PROFILE_AUTO, 0, 0, 0, -1, 0, -1, -1};
  const long shapes[][3] = {""" + ", ".join("{%d, %d, %d}" % s for s in shapes) + r"""};
  for (const auto& s : shapes) {
    const B128Config c = choose_b128(s[0], s[2], (s[1] + 127) / 128, automatic, 152);
    const long tm = 128 * c.cg;
    const long tiles = (s[0] + tm - 1) / tm * ((s[2] + c.bn - 1) / c.bn);
    std::printf("%d %d %d %ld\n", c.cg, c.few, c.splits, tiles);
  }
}
""", "")
    plans = [tuple(map(int, line.split())) for line in out.split("\n") if line]
    long, few = plans[:len(LONG)], plans[len(LONG):]
    assert {p[0] for p in long} == {1, 2} and all(p[1] == 0 for p in long)
    # by either tile, given or chosen, every CTA or pair has two or more
    for (bt, k, n), p in zip(LONG, long):
        assert -(-bt // 256) * -(-n // 256) > 76 and -(-bt // 128) * -(-n // 128) > 152
    assert {p[1] for p in few} == {16, 32, 64, 128}
    assert all(p[2] == 1 and p[3] > 152 for p in few)


def test_norm_shapes_take_their_forms(tmp_path):
    from tests import test_gpu_ops_forms as forms
    warp, block, stream = 0, 1, 2
    want = [(rows, cols, streams, False, stream, 2) for rows, cols in forms.STREAMS
            for streams in (1, 2)]
    want += [(rows, cols, streams, True, stream, 1 if cols <= 8192 else 2)
             for rows, cols in forms.BACKWARD_STREAMS for streams in (2, 3)]
    form = [(warp, 2), (block, 1), (block, 2), (block, 1), (block, 2), (block, 4), (stream, 1),
            (stream, 2), (stream, 1)]
    want += [(rows, cols, 2, False) + f
             for (rows, cols), f in zip(forms.IN_PLACE, form, strict=True)]
    out = run(tmp_path, r"""
#include <cstdio>
#include "forge_norm.cu"
namespace forge {
bool host_map(CUtensorMap*, const void*, CUtensorMapDataType, uint64_t, uint64_t, uint64_t,
              uint32_t, uint32_t, CUtensorMapSwizzle) { return false; }
}
int main() {
  const int shapes[][4] = {""" + ", ".join("{%d, %d, %d, %d}" % w[:4] for w in want) + r"""};
  for (const auto& s : shapes) {
    const forge::RowPlan p = forge::row_plan(s[0], s[1], s[2], s[3], 152);
    std::printf("%d %d %d\n", p.walk, p.vpt, p.direct);
  }
}
""", "", ["-Xptxas", "-O1"])
    got = [tuple(map(int, line.split())) for line in out.split("\n") if line]
    assert got == [w[4:] + (0,) for w in want]


def test_no_memory_for_a_tensor_map_is_no_exception(tmp_path):
    # the cache of tensor maps may not grow: the map is made all the same, and no
    # C++ exception leaves the library (whose callers are C and Python)
    _build.build()
    objects = [os.path.join(_build.BUILD, o) for o in sorted(os.listdir(_build.BUILD))
               if o.endswith(".o") and o != "forge_api.o"]
    run(tmp_path, r"""
#include "forge_api.cu"
extern bool none;   // no memory to be had
static CUresult encode(CUtensorMap* m, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                       const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                       CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                       CUtensorMapFloatOOBfill) {
  m->opaque[0] = 77;
  return CUDA_SUCCESS;
}
int main() {
  forge::g_encode = encode;
  CUtensorMap m;
  for (int i = 0; i < 3; ++i) {
    none = i == 1;
    m.opaque[0] = 0;
    try {
      if (!forge::host_map(&m, &m + i, CU_TENSOR_MAP_DATA_TYPE_UINT8, 128, 128, 128, 128, 128,
                           CU_TENSOR_MAP_SWIZZLE_128B) || m.opaque[0] != 77)
        return 1;
    } catch (...) {
      return 2;
    }
  }
  return 0;
}
""", """
#include <cstdlib>
#include <new>
bool none = false;
void* operator new(std::size_t n, std::align_val_t a) {   // (a tensor map is 64-byte aligned)
  void* p = none ? nullptr : std::aligned_alloc(static_cast<std::size_t>(a), (n + 63) / 64 * 64);
  if (!p) throw std::bad_alloc();
  return p;
}
void operator delete(void* p, std::align_val_t) noexcept { std::free(p); }
void operator delete(void* p, std::size_t, std::align_val_t) noexcept { std::free(p); }
""", objects)


# launches that the program counts; the device has 152 SMs
RUNTIME = """
#include <cuda_runtime_api.h>
#include <atomic>
std::atomic<int> launches{0}, empty{0};
extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t*) {
  *n = 76;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void*, void**) {
  ++(c->gridDim.x > 0 ? launches : empty);
  return cudaSuccess;
}
}
"""
THREADS = """
#include <thread>
#include <vector>
extern std::atomic<int> launches, empty;
template <typename F> int on_threads(F f) {
  std::vector<std::thread> t;
  for (int i = 0; i < 8; ++i) t.emplace_back([&] { for (int k = 0; k < 50; ++k) f(); });
  for (auto& x : t) x.join();
  return launches == 400 && empty == 0 ? 0 : 1;
}
"""


@pytest.mark.parametrize("source,call", [
    ("forge_gemm_b128.cu", "forge::B128Args a = {}; a.num_tiles = 100; "
     "forge::launch_gemm_b128({2, 256, 0, 1}, false, a, 152, nullptr);"),
    ("forge_gemm_b128_few.cu", "forge::B128Args a = {}; a.num_tiles = 100; a.splits = 1; "
     "forge::launch_gemm_b128_few(16, true, a, 152, nullptr);"),
    ("forge_norm.cu", "forge::NormArgs a = {}; a.rows = 8192; a.cols = 4096; "
     "forge::launch_rmsnorm(a, 152, nullptr);"),
])
def test_first_calls_from_several_threads(tmp_path, source, call):
    # what a launch works out once per device is shared by threads: the thread
    # sanitizer must see no race, and no launch may be without blocks
    with open(os.path.join(tmp_path, "t.cpp"), "w") as f:
        f.write("int main() { return 0; }")
    if shutil.which("g++") is None or subprocess.run(
            ["g++", "-fsanitize=thread", f.name, "-o", f.name + ".exe"],
            capture_output=True).returncode:
        pytest.skip("no thread sanitizer")
    run(tmp_path, f"""
#include <atomic>
#include "{source}"
{THREADS}
namespace forge {{
bool host_map(CUtensorMap*, const void*, CUtensorMapDataType, uint64_t, uint64_t, uint64_t,
              uint32_t, uint32_t, CUtensorMapSwizzle) {{ return true; }}
}}
int main() {{ return on_threads([] {{ {call} }}); }}
""", RUNTIME, ["-Xcompiler", "-fsanitize=thread", "-Xptxas", "-O1"])
