"""Where the product of 16-bit x copies its rows from (csrc/mx_tile.hpp), on the
host: every 16 bytes lie inside x, and are the right ones wherever they are used."""
import os
import subprocess

import pytest

from weight_only_quantized_msd_amd import build as B

PROGRAM = r"""
#include <cstdio>
#include "mx_tile.hpp"
using namespace wqbmm;

// A tile of BM rows, four waves of BM / 16 pieces of four rows each; `rows` of them
// exist, of K values, ld values apart.
static int check(int BM, int rows, int K, int64_t ld) {
  const int blocks = K / 32, kt_end = (K + 127) / 128;
  const int64_t bytes = ((rows - 1) * ld + K) * 2;
  for (int kt = 0; kt < kt_end; ++kt)
    for (int piece = 0; piece < BM / 4; ++piece)
      for (int lane = 0; lane < 64; ++lane) {
        const int row = 4 * piece + lane / 16, chunk = lane % 16 ^ (row & 15);
        const int left = kt < blocks / 4 ? 4 : blocks % 4;        // blocks of the K-tile
        const int64_t at = (int64_t)mx_x_row(row, rows, ld) + mx_x_chunk(chunk, left);
        const int64_t from = at + 256 * kt;
        const bool used = row < rows && chunk < 4 * left;
        // the lane's part alone lies inside as well, whichever of the two a limit is held against
        if (at < 0 || at >= bytes || from % 16 != 0 || from + 16 > bytes ||
            (used && from != row * ld * 2 + kt * 256 + chunk * 16)) {
          std::printf("BM %d rows %d K %d ld %lld kt %d piece %d lane %d: %lld of %lld\n", BM, rows, K, (long long)ld, kt,
                      piece, lane, (long long)from, (long long)bytes);
          return 1;
        }
      }
  return 0;
}

int main() {
  for (int BM : {64, 128})
    for (int rows = 1; rows <= BM; ++rows)
      for (int K = 32; K <= 32 * 13; K += 32)
        for (int64_t ld : {(int64_t)K, (int64_t)K + 8, (int64_t)K + 72, ((int64_t)1 << 22) - 8})
          if (check(BM, rows, K, ld)) return 1;
  return check(128, 127, 1 << 20, ((int64_t)1 << 22) - 8) || check(64, 3, (1 << 20) - 96, (1 << 20) - 96);
}
"""


def test_copies_of_x_stay_inside_it(tmp_path):
    if not os.path.exists(B.HIPCC):
        pytest.skip("no hipcc")
    source, program = tmp_path / "addresses.cpp", str(tmp_path / "addresses")
    source.write_text(PROGRAM)
    r = subprocess.run([B.HIPCC, "-x", "hip", "--offload-arch=gfx950", "-O2", "-std=c++17", "-w", "-I", B.CSRC,
                        str(source), "-o", program], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([program], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
