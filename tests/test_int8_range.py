"""Bounds of the int8 x int8 operators that need no GPU: what a wave reads of LDS, sizes
at the ends of their types."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

ROWS = r"""
#include <cstdio>
#include "w8a8_internal.h"
// every wave's first batch (bt = wave % S; later ones are taken while they exist), for
// every length that a few tokens' codes can have in LDS
template <int U, int S> int bad() {
  int n = 0;
  for (int ldk = 1024; ldk <= 65536; ldk += 1024)
    for (int bt = 0; bt < S; ++bt)
      for (int u = 0; u < U; ++u) {
        const int k = (bt * U + u) * 1024;
        if (!qmm::rows_step_exists<S>(k, u, ldk)) break;
        if (k + 1024 > ldk) ++n;
      }
  return n;
}
int main() {
  std::printf("%d\n", bad<2, 4>() + bad<4, 1>() + bad<2, 1>() + bad<1, 1>());
}
"""


def test_waves_without_a_batch_read_nothing(tmp_path):
    src, exe = tmp_path / "rows.cpp", str(tmp_path / "rows")
    src.write_text(ROWS)
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    r = subprocess.run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", f"-I{rocm}/include",
                        "-I" + os.path.join(ROOT, "gemv_only_quant_amd", "csrc"), str(src), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.strip() == "0", out.stdout
