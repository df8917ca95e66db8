"""Host code of the operators between the 16-bit products that no call reaches without a
device: small programs compiled against its sources (no device is touched)."""
import os
import shutil
import subprocess

import pytest

from tests.test_host_code import RUNTIME, THREADS, run

# the host side with nothing behind it
API = """
#include "forge_api_layer.cu"
namespace forge {
int host_device(HostDevice*) { return 0; }
int host_drop_flag() { return 0; }
bool host_map(CUtensorMap*, const void*, CUtensorMapDataType, uint64_t, uint64_t, uint64_t,
              uint32_t, uint32_t, CUtensorMapSwizzle) { return false; }
cudaError_t linear_few_clusters(int, int, int, int*) { return cudaSuccess; }
cudaError_t launch_gemm_linear(const LinearArgs&, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_gemm_linear_few(int, const LinearArgs&, int, cudaStream_t) { return cudaSuccess; }
int epilogue_bwd_rows(int64_t, int64_t, int) { return 0; }
cudaError_t launch_epilogue_bwd(const EpiBwdArgs&, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_dropout(const uint16_t*, const uint16_t*, uint16_t*, int64_t, int64_t,
                           const DropArgs&, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_rope(const RopeArgs&, int, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_qk_norm_rope(const RopeArgs&, int, cudaStream_t) { return cudaSuccess; }
int qk_bwd_blocks(int) { return 0; }
cudaError_t launch_qk_norm_rope_bwd(const RopeArgs&, int, cudaStream_t) { return cudaSuccess; }
}  // namespace forge
extern "C" void forge_get_tuning(forge_tuning*) {}
"""


def test_views_that_share_an_element_are_found(tmp_path):
    # against a search through all elements; views that are only interleaved rows of one
    # buffer must pass
    run(tmp_path, "#include <cstdio>\n#include <set>\n" + API + r"""
int main() {
  static uint16_t buf[1 << 14];
  int apart = 0, missed = 0, together = 0;
  uint64_t seed = 1;
  auto rnd = [&](int n) {
    seed = seed * 6364136223846793005ull + 1442695040888963407ull;
    return static_cast<int>((seed >> 33) % n);
  };
  for (int i = 0; i < 60000; ++i) {
    const int64_t dim = 8 * (1 + rnd(2));
    View v[2];
    std::set<int64_t> at[2];
    const int64_t tokens = 1 + rnd(4), row = 8 * (2 + rnd(16));
    for (int k = 0; k < 2; ++k) {
      const int64_t heads = 1 + rnd(4), first = 8 * rnd(64);
      const bool same = rnd(3) > 0;
      v[k] = View(buf + first, same ? row : 8 * rnd(40), rnd(3) ? dim : 8 * rnd(12), tokens, heads, dim);
      for (int64_t t = 0; t < tokens; ++t)
        for (int64_t h = 0; h < heads; ++h)
          for (int64_t j = 0; j < dim; ++j) at[k].insert(first + t * v[k].token + h * v[k].head + j);
    }
    bool share = false;
    for (int64_t e : at[0]) share |= at[1].count(e) > 0;
    const bool said = views_meet(v[0], v[1]);
    if (share && !said) {
      std::printf("missed: %d\n", i);
      return 1;
    }
    together += share;
    apart += !share && !said;
    missed += !share && said;
  }
  std::printf("%d share, %d apart, %d apart and refused\n", together, apart, missed);
  return together > 1000 && apart > 1000 ? 0 : 2;
}
""", "")


def test_an_output_has_no_element_twice(tmp_path):
    run(tmp_path, "#include <cstdio>\n#include <set>\n" + API + r"""
int main() {
  alignas(16) static uint16_t buf[8];
  int fine = 0, refused = 0;
  for (int64_t dim : {8, 16})
    for (int64_t tokens = 1; tokens <= 4; ++tokens)
      for (int64_t heads = 1; heads <= 4; ++heads)
        for (int64_t ts = 0; ts <= 96; ts += 8)
          for (int64_t hs = 0; hs <= 96; hs += 8) {
            const View v(buf, ts, hs, tokens, heads, dim);
            std::set<int64_t> at;
            for (int64_t t = 0; t < tokens; ++t)
              for (int64_t h = 0; h < heads; ++h)
                for (int64_t j = 0; j < dim; ++j) at.insert(t * v.token + h * v.head + j);
            const bool once = static_cast<int64_t>(at.size()) == tokens * heads * dim;
            const bool ok = check_view(v, true) == FORGE_OK;
            if (ok && !once) return 1;
            fine += ok;
            refused += !ok && !once;
          }
  return fine > 500 && refused > 500 ? 0 : 2;
}
""", "")


def test_product_shapes_take_their_forms(tmp_path):
    # on 152 SMs: single CTAs for few tokens and small outputs, with every split there is,
    # and pairs of every width; a split has two steps a CTA at least, all resident at once;
    # more tiles of 65 to 128 tokens than SMs are pairs'
    out = run(tmp_path, "#include <cstdio>\n" + API + r"""
int main() {
  const forge_tuning automatic = {FORGE_PROFILE_AUTO, 0, 0, 0, -1, 0, -1, -1};
  const int clusters[4] = {152, 76, 36, 16};
  for (int64_t m : {1, 16, 17, 40, 100, 128, 129, 200, 333, 512, 1000, 2000, 4096, 8192})
    for (int64_t n : {8, 136, 520, 1024, 2080, 4096, 14336, 40000})
      for (int64_t k : {8, 136, 1032, 4096, 14336}) {
        const int64_t kb = (k + 63) / 64;
        const LinearConfig c = choose_linear(m, n, kb, automatic, 152, clusters);
        const int64_t tiles = (n + 127) / 128 * ((m + 127) / 128);
        if (c.few) {
          if (c.few < (m < 128 ? m : 128) || c.bn != 128) return 1;
          int i = 0;
          while (1 << i < c.splits) ++i;
          if (c.splits > 1 && (kb < 2 * c.splits || tiles > clusters[i])) return 2;
          if (m > 64 && m <= 128 && tiles > 152) return 4;
        } else if ((m <= 128 && (m <= 64 || tiles <= 152)) || c.bn % 32 || c.bn < 64 ||
                   c.bn > 256 || c.splits != 1) {
          return 3;
        }
        for (int bn : {0, 64, 256}) {   // a limit on the width holds whatever is asked for
          forge_tuning asked = automatic;
          asked.cta_group = 2;
          asked.bn = bn;
          const LinearConfig w = choose_linear(m, n, kb, asked, 152, clusters, 192);
          if (w.few || w.bn > 192 || (bn && w.bn != (bn < 192 ? bn : 192))) return 5;
        }
        std::printf("%d %d %d\n", c.few, c.bn, c.splits);
      }
  return 0;
}
""", "")
    plans = {tuple(map(int, line.split())) for line in out.split("\n") if line}
    assert {p[0] for p in plans} == {0, 16, 32, 64, 128}
    assert {p[2] for p in plans if p[0]} == {1, 2, 4, 8}
    assert len({p[1] for p in plans if not p[0]}) >= 4


def test_columns_of_the_last_tile_stay_in_32_bits(tmp_path):
    # outputs are counted in 32-bit numbers: a width of which no whole number of tiles ends at
    # 2^31 must not be taken where the last tile would reach behind it
    run(tmp_path, "#include <cstdio>\n" + API + r"""
int main() {
  const int clusters[4] = {152, 76, 36, 16};
  int pairs = 0;
  for (int64_t m : {1, 16, 100, 128, 300, 40000})
    for (int64_t less = 8; less <= 512; less += 8)
      for (int cg : {0, 1, 2})
        for (int bn : {0, 128, 256})
          for (int most : {192, 256})
            for (int64_t kb : {1, 3, 64}) {
              const forge_tuning tune = {FORGE_PROFILE_AUTO, cg, bn, 0, -1, 0, -1, -1};
              const int64_t n = (1LL << 31) - less;
              const LinearConfig c = choose_linear(m, n, kb, tune, 152, clusters, most);
              if ((n + c.bn - 1) / c.bn * c.bn > 1LL << 31) {
                std::printf("%lld outputs in tiles of %d\n", static_cast<long long>(n), c.bn);
                return 1;
              }
              pairs += c.few == 0;
            }
  return pairs > 1000 ? 0 : 2;
}
""", "")


@pytest.mark.parametrize("source,call", [
    ("forge_gemm_linear.cu", "forge::LinearArgs a = {}; a.num_tiles = 100; a.e.act = 1; "
     "forge::launch_gemm_linear(a, 152, nullptr);"),
    ("forge_gemm_linear_few.cu", "forge::LinearArgs a = {}; a.num_tiles = 10; a.num_kb = 9; "
     "a.splits = 4; forge::launch_gemm_linear_few(16, a, 152, nullptr);"),
])
def test_first_calls_from_several_threads(tmp_path, source, call):
    # what a launch works out once per device is shared by threads: the thread sanitizer
    # must see no race, and no launch may be without blocks
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
int main() {{ return on_threads([] {{ {call} }}); }}
""", RUNTIME, ["-Xcompiler", "-fsanitize=thread", "-Xptxas", "-O1"])
