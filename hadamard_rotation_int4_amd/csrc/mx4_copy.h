// Where the copies of mx4_gemm_tile_kernel read: offsets into a buffer that holds the
// rows of a tile's operand and no more.
//
// A copy adds a vector offset (a lane's) and a scalar one (the wave's) to the buffer's
// base.  The buffer's range check is only sure to see the vector offset, so that alone
// decides whether a lane reads: below the buffer's size, vector and scalar offset
// together stay in the lane's own row; at or past it the lane reads nothing.  So rows
// are counted in the vector offset and bytes along a row in the scalar one.
// (constexpr, for the host to check.)
#pragma once

namespace hr {

constexpr int kMxStageBytes = 128;       // of a row: 256 codes, 8 blocks
constexpr int kNowhere = 0x40000000;     // past the end of every panel of an operand

// Stages of 8 blocks.
constexpr int mx4_stages(int blocks) { return (blocks + 7) / 8; }

// Codes: 8 rows an instruction, 8 lanes a row, 16 bytes a lane; the scalar offset of
// stage s is s * kMxStageBytes.  Lane l writes place l % 8 of row l / 8, which holds
// chunk l % 8 ^ row / 2 % 8; `odd` is bit 0 of row / 8.
constexpr int mx4_chunk(int lane, int odd) { return (lane & 7) ^ ((lane >> 4) + 4 * odd); }

// Vector offset of this lane in a copy whose first row is 0: of any stage but the last;
// of the last one, in which chunks past the end take the row's last one.
constexpr int mx4_lane_offset(int lane, int odd, int blocks) {
  return (lane >> 3) * (16 * blocks) + 16 * mx4_chunk(lane, odd);
}
constexpr int mx4_lane_offset_last(int lane, int odd, int blocks) {
  const int chunk = mx4_chunk(lane, odd), last = blocks - 1 - 8 * (mx4_stages(blocks) - 1);
  return (lane >> 3) * (16 * blocks) + 16 * (chunk < last ? chunk : last);
}

// The one to take at stage s; behind the last stage nothing is read.
constexpr int mx4_stage_offset(int s, int stages, int offset, int offset_last) {
  return s < stages - 1 ? offset : s < stages ? offset_last : kNowhere;
}

// Vector offset of the copy that begins at row `row`.
constexpr int mx4_copy_offset(int offset, int row, int blocks) { return offset + row * (16 * blocks); }

// Scales, where a row's are whole runs of 16: 64 rows an instruction, a lane the run of
// stages 2 q and 2 q + 1 of its row; the scalar offset is 16 q.
constexpr int mx4_scale_offset(int lane, int row, int q, int blocks) {
  return (16 * q < blocks ? lane * blocks : kNowhere) + row * blocks;
}

// How many loads of a wave may still be under way when the stage after this one has
// landed: the copies of the depth - 2 stages behind it, `codes` a stage and `scales`
// every second one.  Loads complete in order, so a wait for fewer than these is sure
// to cover everything older.  Copies alone count: a plain load is the compiler's, which may
// drop, join or split it, and one that was counted and is not there would end the wait
// early.  Where there are plain loads as well the wait is longer than it need be, which
// does not show: 512 x 4096 x 4128 15.6 us, with them counted 15.7; 2048 x 4096 x 1152 14.5
// and 14.7.
constexpr int mx4_away(int depth, int codes, int scales) { return (depth - 2) * codes + (depth - 2) / 2 * scales; }
// The same before the first stage, with depth stages on their way.
constexpr int mx4_away_first(int depth, int codes, int scales) {
  return depth > 2 ? mx4_away(depth, codes, scales) + codes : 0;
}

}  // namespace hr
