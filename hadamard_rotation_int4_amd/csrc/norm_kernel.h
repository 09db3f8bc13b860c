// The kernel of what stands between two blocks of a layer: the block's output normed, gated,
// scaled and added to the residual stream, and the new stream normed for the
// next block.
//
// What is computed, for every row of n elements, in fp32:
//   u = o, or post_weight * o / sqrt(mean(o^2) + eps)
//   r = x + scale * gate * u                     (stored in x's type)
//   h = weight * r / sqrt(mean(r^2) + eps)       (from r as computed, not as stored)
// h is rounded once to its type, or goes to MXFP4 (mx4_quant.hip) unrounded,
// rotated on the way if asked.
//
// A row is held by a workgroup, or by 8 to 64 lanes of a wave where it is short, an octet
// of 8 elements a lane and turn, so that every operand is read once.  Workgroups stay for
// many rows: weights are read once up to 8192 elements (for each row past them), and a
// row's operands are asked for before the sums of the row before it, whose waits they
// then hide.
//
// All of a row is in registers up to 8192 elements, and up to 16384 where the result is not
// MXFP4 and stream and block are not both fp32.  Past 8192 a workgroup has 1024 threads of
// 128 registers; what does not fit goes through scratch: up to 16384 elements 8 to 31
// registers, past them 126 to 186, with an fp32 stream and block 513 to 643.
//
// Bound by memory when there are many rows: bf16 16384 x 4096 with a block, its norm
// and a gate takes 92 us (537 MB, 5.8 TB/s, where a large copy reaches 5.3 and one
// operand negated 6.1), to MXFP4 through a rotation 75 (438 MB).  Bound by the launch
// and two sums over the row when there are few: one row of 4096 3.2 us.  By waves, of which
// more than 128 registers leave 3 a SIMD, to MXFP4 at 4097 to 8192 elements: 16384 x 5120
// 205 us where bf16 results take 118.  By rows at odd addresses: 32768 x 2047 205 us where
// 2048 take 96.  By scratch past 16384: 1024 x 32768 119 us (bf16, 268 MB), in fp32 222
// (537 MB).
#pragma once

#include "mx4_device.h"

namespace hr {

// 16 bytes at any address.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// 8 elements of type DT as they lie in memory.
template <int DT>
struct Octet { uint32_t v[DT == kDtF32 ? 8 : 4]; };

// From element `at` of base, which need not be aligned; zeros from the n-th of the
// row on.
template <int DT, bool NT = false>
__device__ __forceinline__ void load_octet(const void* base, int64_t at, int col, int n, Octet<DT>& o) {
  if (col + 8 <= n) {
    const u32x4_any* q = reinterpret_cast<const u32x4_any*>(reinterpret_cast<const char*>(base) + at * (DT == kDtF32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (DT == kDtF32 ? 2 : 1); ++i) {
      const u32x4_any x = NT ? __builtin_nontemporal_load(q + i) : q[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) o.v[4 * i + e] = x[e];
    }
    return;
  }
  if (DT == kDtF32) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      o.v[e] = col + e < n ? reinterpret_cast<const uint32_t*>(base)[at + e] : 0u;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint16_t* q = reinterpret_cast<const uint16_t*>(base) + at + 2 * i;
      const uint32_t lo = col + 2 * i < n ? q[0] : 0u, hi = col + 2 * i + 1 < n ? q[1] : 0u;
      o.v[i] = lo | (hi << 16);
    }
  }
}

template <int DT>
__device__ __forceinline__ void widen(const Octet<DT>& o, float* w) {
#pragma unroll
  for (int i = 0; i < (DT == kDtF32 ? 8 : 4); ++i) {
    if (DT == kDtF32) {
      w[i] = __uint_as_float(o.v[i]);
    } else if (DT == kDtBf16) {
      w[2 * i] = __uint_as_float(o.v[i] << 16);
      w[2 * i + 1] = __uint_as_float(o.v[i] & 0xFFFF0000u);
    } else {
      const half2v h = __builtin_bit_cast(half2v, o.v[i]);
      w[2 * i] = (float)h[0];
      w[2 * i + 1] = (float)h[1];
    }
  }
}

template <int DT, bool NT>
__device__ __forceinline__ void store_octet(void* base, int64_t at, int col, int n, const float* w) {
  if (col + 8 <= n) {
    u32x4_any* q = reinterpret_cast<u32x4_any*>(reinterpret_cast<char*>(base) + at * (DT == kDtF32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (DT == kDtF32 ? 2 : 1); ++i) {
      u32x4_any x;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (DT == kDtF32) x[e] = __float_as_uint(w[4 * i + e]);
        else if (DT == kDtBf16) x[e] = __builtin_bit_cast(uint32_t, (bf16x2){(__bf16)w[2 * e], (__bf16)w[2 * e + 1]});
        else x[e] = __builtin_bit_cast(uint32_t, (half2v){(_Float16)w[2 * e], (_Float16)w[2 * e + 1]});
      }
      if (NT) __builtin_nontemporal_store(x, q + i);
      else q[i] = x;
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (col + e < n) {
      if (DT == kDtF32) reinterpret_cast<float*>(base)[at + e] = w[e];
      else if (DT == kDtBf16) reinterpret_cast<__bf16*>(base)[at + e] = (__bf16)w[e];
      else reinterpret_cast<_Float16*>(base)[at + e] = (_Float16)w[e];
    }
}

// Sum over N consecutive lanes, the same in every one: partners add the same two
// numbers.
template <int N>
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<kQuadXor1>(v);
  v += dpp<kQuadXor2>(v);
  v += dpp<kRowHalfMirror>(v);
  if (N >= 16) v += dpp<kRowMirror>(v);
  if (N >= 32) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  if (N >= 64) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  return v;
}

// Sum over the workgroup, the same in every thread.  Its own barrier waits for LDS
// alone and leaves loads in flight; no two sums that no other lies between may share
// a slot.
template <int WAVES>
__device__ __forceinline__ float block_sum(float v, float (*red)[WAVES], int slot) {
  v = wave_sum<64>(v);
  if (WAVES == 1) return v;
  if ((threadIdx.x & 63) == 0) red[slot][threadIdx.x >> 6] = v;
  __builtin_amdgcn_s_waitcnt(0xC07F);              // lgkmcnt(0)
  mx_barrier();
  float t = 0.0f;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) t += red[slot][w];
  return t;
}

// XT, DT: types of the stream and of the block and the norm; LANES of a row, 64 WAVES
// (a workgroup of WAVES) or fewer (4 waves, each with 64 / LANES rows); CH octets a lane;
// NT: rows are read and written around the L2s; QUANT: h goes to MXFP4.
template <int XT, int DT, int LANES, int CH, bool NT, bool QUANT>
__global__ __launch_bounds__(LANES <= 64 ? 256 : LANES) void norm_kernel(NormArgs p) {
  constexpr int WAVES = LANES <= 64 ? 1 : LANES / 64;      // of a row
  constexpr int ROWS = LANES <= 64 ? 256 / LANES : 1;      // of a workgroup at a time
  __shared__ float red[4][WAVES];
  // the same labels with and without a rotation, so that sums have one order and
  // r the same bits
  const int lane = mx4_lane(threadIdx.x & 63) | (threadIdx.x & ~63);
  const int a = ROWS > 1 ? lane & (LANES - 1) : lane, mine = ROWS > 1 ? lane / LANES : 0;
  auto row_sum = [&](float v, int slot) {
    if constexpr (LANES <= 64) return wave_sum<LANES>(v);
    else return block_sum<WAVES>(v, red, slot);
  };
  int col[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) col[i] = 8 * (a + i * LANES);

  // What rows share: the factors of the norm, with the rotation's signs and scale, and
  // of the block's output; kept where there are registers for them.
  constexpr bool KEEP = LANES * CH <= 1024;
  const bool one_gate = p.gate && p.gate_rows >= p.rows, row_gate = p.gate && !one_gate;
  auto norm_factors = [&](int i, float* w) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = QUANT ? p.turn : 1.0f;
    if (p.weight) {
      Octet<kDtF32> o;
      load_octet<kDtF32>(p.weight, col[i], col[i], p.n, o);
      float v[8];
      widen<kDtF32>(o, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] *= v[e];
    }
    if (QUANT && p.signs) {
      uint32_t sg[8];
      load_signs<8>(p.signs, col[i] < p.n ? col[i] : 0, sg);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = flip(w[e], sg[e]);
    }
  };
  auto block_factors = [&](int i, float* w) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.0f;
    if (p.post_weight) {
      Octet<kDtF32> o;
      load_octet<kDtF32>(p.post_weight, col[i], col[i], p.n, o);
      widen<kDtF32>(o, w);
    }
    if (one_gate) {
      Octet<DT> g;
      float v[8];
      load_octet<DT>(p.gate, col[i], col[i], p.n, g);
      widen<DT>(g, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] *= v[e];
    }
  };
  float wt[KEEP ? CH : 1][8], pw[KEEP ? CH : 1][8];
  if (KEEP) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      norm_factors(i, wt[i]);
      if (p.block) block_factors(i, pw[i]);
    }
  }
  const uint32_t flips = QUANT && p.order && mx4_negated(a, p.order) ? 0x88888888u : 0u;

  Octet<XT> xo[CH];
  Octet<DT> bo[CH], go[CH];
  auto load_row = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      load_octet<XT, NT>(p.x, row * p.x_stride + col[i], col[i], p.n, xo[i]);
      if (p.block) load_octet<DT, NT>(p.block, row * p.block_stride + col[i], col[i], p.n, bo[i]);
      if (row_gate) load_octet<DT>(p.gate, (int64_t)((uint32_t)row / (uint32_t)p.gate_rows) * p.n + col[i], col[i], p.n, go[i]);
    }
  };
  // rows of a turn past the end: the last again, stored nowhere (its elements end at 0)
  const int64_t step = (int64_t)gridDim.x * ROWS;
  auto row_of = [&](int64_t first) { return ROWS > 1 ? (first + mine < p.rows ? first + mine : p.rows - 1) : first; };
  load_row(row_of((int64_t)blockIdx.x * ROWS));
  int slot = 0;
  for (int64_t first = (int64_t)blockIdx.x * ROWS; first < p.rows; first += step) {
    const int64_t row = row_of(first);
    const int end = ROWS == 1 || first + mine < p.rows ? p.n : 0;
    float r[CH][8], u[CH][8];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      widen<XT>(xo[i], r[i]);
      if (p.block) widen<DT>(bo[i], u[i]);
    }
    float sum = 0.0f;
    if (p.block) {
      // the square sum is of the block's output itself, before its gate
      if (p.post_norm) {
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) sum = fmaf(u[i][e], u[i][e], sum);
      }
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        float* const w = pw[KEEP ? i : 0];
        if (!KEEP) block_factors(i, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[i][e] *= w[e];
        if (row_gate) {
          float v[8];
          widen<DT>(go[i], v);
#pragma unroll
          for (int e = 0; e < 8; ++e) u[i][e] *= v[e];
        }
      }
    }
    if (first + step < p.rows) load_row(row_of(first + step));
    if (p.block) {
      float f = p.scale;
      if (p.post_norm) f = p.scale / sqrtf(row_sum(sum, slot) / (float)p.n + p.eps);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) r[i][e] = fmaf(u[i][e], f, r[i][e]);
        store_octet<XT, NT>(p.residual, row * p.residual_stride + col[i], col[i], end, r[i]);
      }
    }
    if (QUANT || p.h) {
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(r[i][e], r[i][e], sum);
      const float f = 1.0f / sqrtf(row_sum(sum, slot + 1) / (float)p.n + p.eps);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        float* const w = wt[KEEP ? i : 0];
        if (!KEEP) norm_factors(i, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[i][e] *= f * w[e];
        if (!QUANT) {
          store_octet<DT, NT>(p.h, row * p.n + col[i], col[i], end, r[i]);
          continue;
        }
        mx4_fwht(r[i], a, p.order);
        const uint32_t b = mx4_scale(mx4_absmax(r[i]), p.ceil);
        const uint32_t code = mx4_codes(r[i], b) ^ (b == 255u ? 0u : flips);
        if (col[i] < end) {
          reinterpret_cast<uint32_t*>(p.codes)[(row * p.n + col[i]) >> 3] = code;
          if ((a & 3) == 0) p.scales[(row * p.n + col[i]) >> 5] = (uint8_t)b;
        }
      }
    }
    slot ^= 2;
  }
}

template <int XT, int DT, int LANES, int CH>
static void launch_rows(const NormArgs& a, hipStream_t s) {
  constexpr int THREADS = LANES <= 64 ? 256 : LANES, ROWS = THREADS / LANES;
  // 16 waves a compute unit, unless that leaves them uneven numbers of few rows
  const int64_t turns = (a.rows + ROWS - 1) / ROWS, most = 256 * 1024 / THREADS;
  const dim3 grid((unsigned)(turns < 4 * most ? turns : most)), threads(THREADS);
  // large streams of aligned rows: 16384 x 4096 bf16 95 us against 102 without the hint, to
  // MXFP4 78 against 88; of rows that share lines, 16384 x 4094 bf16 126 against 116, 16384 x
  // 4095 of an fp32 stream and a bf16 block 186 against 168, of an fp32 block 288 against 264
  const bool nt = a.rows * a.n * (XT == kDtF32 ? 4 : 2) >= kStreamBytes && a.n % 8 == 0;
  if (a.codes) {
    if (nt) hipLaunchKernelGGL((norm_kernel<XT, DT, LANES, CH, true, true>), grid, threads, 0, s, a);
    else hipLaunchKernelGGL((norm_kernel<XT, DT, LANES, CH, false, true>), grid, threads, 0, s, a);
  } else {
    if (nt) hipLaunchKernelGGL((norm_kernel<XT, DT, LANES, CH, true, false>), grid, threads, 0, s, a);
    else hipLaunchKernelGGL((norm_kernel<XT, DT, LANES, CH, false, false>), grid, threads, 0, s, a);
  }
}

// The lanes that a row needs, by its length alone: a row's bits do not depend on how
// many there are.
template <int XT, int DT>
static void launch_length(const NormArgs& a, hipStream_t s) {
  if (a.n <= 64) launch_rows<XT, DT, 8, 1>(a, s);
  else if (a.n <= 128) launch_rows<XT, DT, 16, 1>(a, s);
  else if (a.n <= 256) launch_rows<XT, DT, 32, 1>(a, s);
  else if (a.n <= 512) launch_rows<XT, DT, 64, 1>(a, s);
  else if (a.n <= 1024) launch_rows<XT, DT, 64, 2>(a, s);
  else if (a.n <= 2048) launch_rows<XT, DT, 256, 1>(a, s);
  else if (a.n <= 4096) launch_rows<XT, DT, 256, 2>(a, s);
  else if (a.n <= 8192) launch_rows<XT, DT, 512, 2>(a, s);
  else if (a.n <= 16384) launch_rows<XT, DT, 1024, 2>(a, s);
  else launch_rows<XT, DT, 1024, 4>(a, s);
}

}  // namespace hr
