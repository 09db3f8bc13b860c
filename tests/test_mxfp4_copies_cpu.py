"""Where the MXFP4 product's copies into LDS read, checked on the host for every lane.

A buffer's range check is sure to see a lane's vector offset; whether it counts the
scalar offset too is not relied on.  So for rows 0 .. rows - 1 of `size` bytes each in a
buffer of rows * size bytes, a lane's 16 bytes must be either nowhere (vector offset
at or past the buffer's size) or inside one row, vector and scalar offset together.

A stage waits until at most so many loads are under way.  Loads complete in order; the
copies are certain to be among them, the compiler's plain loads are not, so the wait has
to cover the next stage whether those are there or not.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "hadamard_rotation_int4_amd", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "mx4_copy.h"
using namespace hr;

// one lane's read of a buffer of `rows` rows of `size` bytes; the row it reads, -1 for none
static int read_row(long v, long s, int rows, int size, const char* what, int blocks) {
  const long total = (long)rows * size;
  if (v < 0 || s < 0 || v + s + 16 >= 1L << 31) { std::printf("%s: offset %ld + %ld, blocks %d\n", what, v, s, blocks); std::exit(1); }
  if (v >= total) return -1;
  const long row = v / size;
  if (v + s < row * size || v + s + 16 > (row + 1) * size) {
    std::printf("%s: offsets %ld + %ld leave row %ld of %d rows of %d bytes\n", what, v, s, row, rows, size);
    std::exit(1);
  }
  return (int)row;
}

int main(int argc, char** argv) {
  const int tile = std::atoi(argv[1]);
  for (int i = 2; i < argc; ++i) {
    const int blocks = std::atoi(argv[i]), stages = mx4_stages(blocks);
    for (int rows : {1, 2, 7, 8, 9, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256}) {
      if (rows > tile) break;
      std::vector<char> seen((size_t)rows * blocks, 0);
      // two teams of four stages in LDS ask for at most 11 stages behind the last one
      for (int s = 0; s < stages + 12; ++s)
        for (int row = 0; row < tile; row += 8)
          for (int lane = 0; lane < 64; ++lane) {
            const int odd = row / 8 & 1, at = row + lane / 8, place = lane & 7;
            const int v = mx4_copy_offset(mx4_stage_offset(s, stages, mx4_lane_offset(lane, odd, blocks),
                                                           mx4_lane_offset_last(lane, odd, blocks)), row, blocks);
            const int got = read_row(v, (long)s * kMxStageBytes, rows, 16 * blocks, "codes", blocks);
            const int chunk = place ^ (at / 2 & 7), block = 8 * s + chunk;
            if (got != (at < rows && s < stages ? at : -1)) { std::printf("codes of row %d\n", at); return 1; }
            if (got < 0) continue;
            // its own chunk, or behind the end of the row the last one
            const long want = (long)at * 16 * blocks + 16 * (block < blocks ? block : blocks - 1);
            if (v + (long)s * kMxStageBytes != want) { std::printf("chunk %d of row %d\n", block, at); return 1; }
            if (block < blocks) seen[(size_t)at * blocks + block] = 1;
          }
      for (char c : seen)
        if (!c) { std::printf("codes never read\n"); return 1; }
      if (blocks % 16) continue;
      for (int q = 0; q < blocks / 16 + 8; ++q)
        for (int row = 0; row < tile; row += 64)
          for (int lane = 0; lane < 64; ++lane) {
            const int got = read_row(mx4_scale_offset(lane, row, q, blocks), 16L * q, rows, blocks, "scales", blocks);
            if (got != (row + lane < rows && q < blocks / 16 ? row + lane : -1)) { std::printf("scales of row %d\n", row + lane); return 1; }
          }
    }
  }
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
@pytest.mark.parametrize("tile", [32, 64, 128, 256])
def test_copies_stay_in_their_rows(tmp_path, tile):
    src, exe = tmp_path / "copies.cpp", tmp_path / "copies"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    # one to 40 blocks, and the longest rows (2^18 elements) with a ragged end and without
    blocks = [*range(1, 41), 64, 95, 96, 100, 256] + ([8190, 8192] if tile < 256 else [8192])
    r = subprocess.run([str(exe), str(tile), *map(str, blocks)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


WAITS = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "mx4_copy.h"
using namespace hr;

int main(int argc, char** argv) {
  const int depth = std::atoi(argv[1]), codes = std::atoi(argv[2]), scales = std::atoi(argv[3]), plain = std::atoi(argv[4]);
  // loads in the order in which a wave issues them: stage s as s, scales of stages 2 i and
  // 2 i + 1 as 1000 + i, plain loads as -1
  std::vector<int> sent;
  auto load = [&](int what, int n) { sent.insert(sent.end(), n, what); };
  auto landed = [&](int away, int what) {
    for (size_t i = sent.size() > (size_t)away ? sent.size() - away : 0; i < sent.size(); ++i)
      if (sent[i] == what) { std::printf("%d is under way\n", what); std::exit(1); }
  };
  load(-1, plain);
  load(0, codes);
  load(1000, scales);
  for (int s = 1; s < depth; ++s) {
    load(s, codes);
    load(-1, plain);
    if (s % 2 == 0) load(1000 + s / 2, scales);
  }
  landed(mx4_away_first(depth, codes, scales), 0);
  landed(mx4_away_first(depth, codes, scales), 1000);
  for (int k = 0; k < 40; ++k) {
    load(-1, plain);
    const int away = mx4_away(depth, codes, scales);
    landed(away, k + 1);
    if (k % 2 == 1) landed(away, 1000 + (k + 1) / 2);
    load(-1, plain);
    load(k + depth, codes);
    if (k % 2 == 0) load(1000 + k / 2 + depth / 2, scales);
  }
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_waits_cover_the_next_stage(tmp_path):
    src, exe = tmp_path / "waits.cpp", tmp_path / "waits"
    src.write_text(WAITS)
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    for depth in (2, 4):
        for codes in (2, 4, 6, 8, 12):
            for scales in (0, 1, 2, 4):
                for plain in (0, 1, 3, 8):
                    r = subprocess.run([str(exe), *map(str, (depth, codes, scales, plain))], capture_output=True, text=True)
                    assert r.returncode == 0, (depth, codes, scales, plain, r.stdout)
