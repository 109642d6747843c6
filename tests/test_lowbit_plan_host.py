"""The division by which the attention's workgroups find their share of all
pages, at every size that the host accepts, on the CPU."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = "/opt/rocm/bin/hipcc"

DIVISION = r"""
#include <hip/hip_runtime.h>
#include <cmath>
#include <cstdio>
#include <random>
#include "sv_cache4.hpp"
static int bad = 0;
static void one(int64_t x, int64_t y) {
  // the hardware's reciprocal is some value near 1 / y; any within 2^-14 has to do
  for (double off : {-0x1p-14, -0x1p-27, 0.0, 0x1p-40, 0x1p-14}) {
    const int64_t got = sv::c4_quotient(x, y, 1.0 / (double)y * (1.0 + off));
    if (got != x / y && bad++ < 5) std::printf("%lld / %lld = %lld\n", (long long)x, (long long)y, (long long)got);
  }
}
int main() {
  const int64_t top = int64_t(1) << 40;
  // places of a call with one kv head and one block of rows are divided by 1; 65,536 sequences of
  // 32,768 pages have 2,148,007,936 of them
  for (int64_t x : {int64_t(2148007936), (int64_t(1) << 31) - 1, int64_t(1) << 31, (int64_t(1) << 39) + 12345, top - 1}) one(x, 1);
  // a share of all places over 512 workgroups reaches 2^31
  const int64_t share = (top - 1 + 511) / 512;
  for (int64_t k = 0; k < 512; ++k) for (int64_t d : {-1, 0, 1}) if (k * share + d >= 0) one(k * share + d, share);
  std::mt19937_64 g(1);
  for (int i = 0; i < 1000000; ++i) {
    const int64_t y = 1 + (int64_t)(g() >> (24 + g() % 40)), q = (int64_t)(g() % (top / y + 1));
    for (int64_t x : {q * y - 1, q * y, q * y + (int64_t)(g() % y)}) if (x >= 0 && x < top) one(x, y);
  }
  std::printf(bad ? "bad %d\n" : "division ok\n", bad);
  return bad != 0;
}
"""


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="no ROCm toolchain")
def test_places_and_shares_past_32_bits(tmp_path):
    src, exe = tmp_path / "t.hip", str(tmp_path / "t")
    src.write_text(DIVISION)
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", "-w",
                        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I",
                        os.path.join(ROOT, "draft_token_verification_11_amd", "csrc"), "-o", exe, str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([exe], capture_output=True, text=True)
    assert "division ok" in out.stdout, out.stdout
