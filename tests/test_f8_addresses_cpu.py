"""Address arithmetic of the F8 tile kernels, evaluated by the compiler (no GPU):
static assertions on the functions that the kernels call."""
import os
import shutil
import subprocess

import pytest

from weight_only_quantized_w8a16_amd import build

pytestmark = pytest.mark.skipif(shutil.which(build.HIPCC) is None, reason="needs hipcc")


def assert_compiles(tmp_path, text):
    src = tmp_path / "addresses.hip"
    src.write_text('#include "f8_tile.hpp"\nusing namespace qg;\n' + text)
    cmd = [build.HIPCC, "-std=c++17", f"--offload-arch={build.ARCH}", "--offload-host-only", "-fsyntax-only",
           "-fconstexpr-steps=100000000", "-I", build.CSRC, "-I", os.path.join(build.ROOT, "include"), str(src)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr


def test_loads_stay_within_the_rows_that_are_left(tmp_path):
    """Every 16 bytes that a wave's four loads ask for pass a bounds check of the vector offset alone (against
    the bytes from here to the end of the last row that is left) if and only if they are a chunk of one of these
    rows, and hold the chunk that the reads look for there."""
    assert_compiles(tmp_path, r'''
constexpr bool holds(uint32_t K, int k0, int rows) {
  const uint32_t bytes = static_cast<uint32_t>(rows) * K - static_cast<uint32_t>(k0);
  const int rem = static_cast<int>(K) - k0;
  for (int lane = 0; lane < 64; ++lane) {
    const F8LaneLoads l(lane, K);
    for (int i = 0; i < 4; ++i) {
      const int row = 8 * i + lane / 8, place = lane % 8, chunk = place ^ ((row / 2) % 8);
      const uint32_t at = l.start(i & 1, rem) + F8LaneLoads::past(i, K);
      const bool wanted = row < rows && 16 * chunk < rem;
      if ((at < bytes) != wanted) return false;
      if (wanted && at != static_cast<uint32_t>(row) * K + 16u * chunk) return false;
    }
  }
  return true;
}
constexpr bool all(uint32_t K, int k0) {
  for (int rows = 1; rows <= 32; ++rows)
    if (!holds(K, k0, rows)) return false;
  return true;
}
static_assert(all(16, 0) && all(112, 0) && all(128, 0) && all(272, 0) && all(272, 256) && all(3584, 3456), "rows");
// the longest rows that the tiles take: 256 of them below 2^31 bytes
static_assert(all((1u << 23) - 16, 0) && all((1u << 23) - 16, (1 << 23) - 128), "long rows");
''')


def test_scales_past_32_bits(tmp_path):
    assert_compiles(tmp_path, r'''
static_assert(f8_scale_offset(1, 1u << 30) * sizeof(float) == size_t(1) << 32, "2^30 rows");
static_assert(f8_scale_offset(3, (1u << 31) - 256) == 3 * ((size_t(1) << 31) - 256), "the most rows");
''')
