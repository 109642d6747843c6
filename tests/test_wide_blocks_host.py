"""How the waves of a workgroup divide a block's rows, and where two waves that have the same rows hand
them over in shared memory, for every size of a block, on the CPU."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = "/opt/rocm/bin/hipcc"

# Each tile of 16 rows of a block belongs to one wave, or one pair of waves; what the pairs hand over,
# O [tiles][D / 16][64 lanes] float4s in the two pages' buffers and m, l, n [tiles][3][64] floats, lies
# apart from what the other pairs do and inside its array.
BLOCKS = r"""
#include <hip/hip_runtime.h>
#include <cstdio>
#include <vector>
#include "sv_cache4_wide.hpp"
static int bad = 0, pairs = 0, uneven = 0;
static void take(std::vector<int>& used, int at, int n, const char* what, int D, int tiles, int w) {
  for (int x = at; x < at + n; ++x)
    if (x < 0 || x >= (int)used.size() || used[x]++) {
      if (bad++ < 8) std::printf("heads of %d, %d tiles, wave %d: %s %d\n", D, tiles, w, what, x);
      return;
    }
}
template <int D>
static void blocks() {
  using Sh = sv::C4Wide<D>;
  for (int rows = 1; rows <= Sh::kRows; ++rows) {
    std::vector<int> tiles((rows + 15) / 16), o(4 * Sh::kKeys / 16), stats(Sh::kStats);
    const bool half = sv::c4_wave_share<D>(rows, 0).half;
    int least = Sh::RT, most = 0;
    for (int w = 0; w < Sh::kWaves; ++w) {
      const sv::C4Share x = sv::c4_wave_share<D>(rows, w);
      if (x.half != half || x.tiles != (int)tiles.size() || x.mine > Sh::RT || x.row0 % 16) ++bad;
      if (half && w % 2 == 0) continue;  // as the next one, which hands over
      take(tiles, x.row0 / 16, x.mine, "tile", D, x.tiles, w);
      if (!half || x.mine == 0) continue;
      ++pairs;
      least = x.mine < least ? x.mine : least, most = x.mine > most ? x.mine : most;
      const sv::C4HandOver a = sv::c4_hand_over<D>(w), b = sv::c4_hand_over<D>(w - 1);
      if (a.o != b.o || a.stats != b.stats) ++bad;
      take(o, a.o, x.mine * (D / 16) * 64, "float4 of O", D, x.tiles, w);
      take(stats, a.stats, x.mine * 3 * 64, "statistic", D, x.tiles, w);
    }
    uneven += half && least != most;
    for (int n : tiles) bad += n != 1;
  }
}
int main() {
  blocks<128>();
  blocks<256>();
  std::printf(bad || !pairs || !uneven ? "bad %d\n" : "blocks ok\n", bad);
  return bad != 0;
}
"""


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="no ROCm toolchain")
def test_rows_and_hand_overs_lie_apart(tmp_path):
    src, exe = tmp_path / "t.hip", str(tmp_path / "t")
    src.write_text(BLOCKS)
    r = subprocess.run([HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", "-w",
                        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I",
                        os.path.join(ROOT, "draft_token_verification_11_amd", "csrc"), "-o", exe, str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    out = subprocess.run([exe], capture_output=True, text=True)
    assert "blocks ok" in out.stdout, out.stdout
