"""Bounds of the int8 x int8 operators that need no GPU: what a wave reads of LDS, sizes
at the ends of their types."""
import os
import subprocess

import pytest
import torch

qmm = pytest.importorskip("gemv_only_quant_amd")
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


def test_sizes_beyond_the_c_types_are_refused():
    """Tensors of 2^31 rows and more (on the meta device: no memory): the C functions take
    ints, and a size that is not one may not arrive as another."""
    big = (1 << 32) + 4
    m = lambda *s, t=torch.int8: torch.empty(s, dtype=t, device="meta")  # noqa: E731
    f, h = torch.float32, torch.float16
    w, s = m(32, 16), m(32, t=f)
    for call in (lambda: qmm.quantize_tokens(m(big, 16, t=h)),
                 lambda: qmm.w8a8_gemm(m(big, 16, t=h), w, s),
                 lambda: qmm.w8a8_gemm(m(big, 16), w, s, sx=m(big, t=f)),
                 lambda: qmm.w8a8_gemm(m(4, 16, t=h), m(big, 16), m(big, t=f)),
                 lambda: qmm.w8a8_gemm(m(4, big, t=h), m(32, big), s),
                 lambda: qmm.w8a8_gated(m(big, 16, t=h), w, s, w, s),
                 lambda: qmm.w8a8_gemm_backward(m(big, 32, t=h), None, None, w, s, weight_grad=False),
                 lambda: qmm.w8a8_gated_backward(m(big, 32, t=h), m(big, 16), m(big, t=f), w, s, w, s)):
        with pytest.raises(qmm.QmmError) as e:
            call()
        assert e.value.status == qmm.QMM_ERR_UNSUPPORTED and "too large" in str(e.value), str(e.value)
