// What stands between two blocks of a layer: the block's output normed, gated,
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
// A row is held in registers by one workgroup, an octet of 8 elements a lane and
// turn, so that every operand is read once.  Workgroups stay for many rows: weights
// are read once, and a row's operands are asked for before the sums of the row before
// it, whose waits they then hide.
#include "mx4_device.h"

namespace hr {

// 8 elements of type DT as they lie in memory.
template <int DT>
struct Octet { uint32_t v[DT == kDtF32 ? 8 : 4]; };

// From element `at` of base, which need not be aligned; zeros from the n-th of the
// row on.
template <int DT>
__device__ __forceinline__ void load_octet(const void* base, int64_t at, int col, int n, Octet<DT>& o) {
  if (col + 8 <= n) {
    struct __attribute__((packed, aligned(DT == kDtF32 ? 4 : 2))) U { Octet<DT> o; };
    o = reinterpret_cast<const U*>(reinterpret_cast<const char*>(base) + at * (DT == kDtF32 ? 4 : 2))->o;
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

template <int DT>
__device__ __forceinline__ void store_octet(void* base, int64_t at, int col, int n, const float* w) {
  if (col + 8 <= n) {
    if (DT == kDtF32) {
      struct __attribute__((packed, aligned(4))) U { float v[8]; };
      U u;
#pragma unroll
      for (int e = 0; e < 8; ++e) u.v[e] = w[e];
      *reinterpret_cast<U*>(reinterpret_cast<float*>(base) + at) = u;
    } else {
      struct __attribute__((packed, aligned(2))) U { uint32_t v[4]; };
      U u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (DT == kDtBf16) {
          const bf16x2 b = {(__bf16)w[2 * i], (__bf16)w[2 * i + 1]};
          u.v[i] = __builtin_bit_cast(uint32_t, b);
        } else {
          const half2v h = {(_Float16)w[2 * i], (_Float16)w[2 * i + 1]};
          u.v[i] = __builtin_bit_cast(uint32_t, h);
        }
      }
      *reinterpret_cast<U*>(reinterpret_cast<uint16_t*>(base) + at) = u;
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

// Sum over the workgroup, the same in every thread.  Its own barrier waits for LDS
// alone and leaves loads in flight; no two sums that no other lies between may share
// a slot.
template <int WAVES>
__device__ __forceinline__ float block_sum(float v, float (*red)[WAVES], int slot) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  if (WAVES == 1) return v;
  if ((threadIdx.x & 63) == 0) red[slot][threadIdx.x >> 6] = v;
  __builtin_amdgcn_s_waitcnt(0xC07F);              // lgkmcnt(0)
  mx_barrier();
  float t = 0.0f;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) t += red[slot][w];
  return t;
}

// XT, DT: types of the stream and of the block and the norm; CH octets a lane;
// L = 0: no rotation, QUANT: h goes to MXFP4.
template <int XT, int DT, int WAVES, int CH, bool QUANT, int L>
__global__ __launch_bounds__(64 * WAVES) void norm_kernel(NormArgs p) {
  __shared__ float red[4][WAVES];
  // the same labels with and without a rotation, so that sums have one order and
  // r the same bits
  const int a = mx4_lane<16>(threadIdx.x & 63) | (threadIdx.x & ~63);
  int col[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) col[i] = 8 * (a + i * 64 * WAVES);

  // What rows share: the factors of the norm, with the rotation's signs and scale, and
  // of the block's output; kept where there are registers for them.
  constexpr bool KEEP = CH <= 2;
  const bool one_gate = p.gate && p.gate_rows >= p.rows, row_gate = p.gate && !one_gate;
  auto norm_factors = [&](int i, float* w) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = L ? mx4_norm<L ? L : 4>() : 1.0f;
    if (p.weight) {
      Octet<kDtF32> o;
      load_octet<kDtF32>(p.weight, col[i], col[i], p.n, o);
      float v[8];
      widen<kDtF32>(o, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] *= v[e];
    }
    if (L) {
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
  const uint32_t flips = L && mx4_negated<L ? L : 4>(a) ? 0x88888888u : 0u;

  Octet<XT> xo[CH];
  Octet<DT> bo[CH], go[CH];
  auto load_row = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      load_octet<XT>(p.x, row * p.x_stride + col[i], col[i], p.n, xo[i]);
      if (p.block) load_octet<DT>(p.block, row * p.block_stride + col[i], col[i], p.n, bo[i]);
      if (row_gate) load_octet<DT>(p.gate, (int64_t)((uint32_t)row / (uint32_t)p.gate_rows) * p.n + col[i], col[i], p.n, go[i]);
    }
  };
  load_row(blockIdx.x);
  int slot = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
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
    if (row + gridDim.x < p.rows) load_row(row + gridDim.x);
    if (p.block) {
      float f = p.scale;
      if (p.post_norm) f = p.scale / sqrtf(block_sum<WAVES>(sum, red, slot) / (float)p.n + p.eps);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) r[i][e] = fmaf(u[i][e], f, r[i][e]);
        store_octet<XT>(p.residual, row * p.residual_stride + col[i], col[i], p.n, r[i]);
      }
    }
    if (QUANT || p.h) {
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(r[i][e], r[i][e], sum);
      const float f = 1.0f / sqrtf(block_sum<WAVES>(sum, red, slot + 1) / (float)p.n + p.eps);
#pragma unroll
      for (int i = 0; i < CH; ++i) {
float* const w = wt[KEEP ? i : 0];
        if (!KEEP) norm_factors(i, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[i][e] *= f * w[e];
        if (!QUANT) {
          store_octet<DT>(p.h, row * p.n + col[i], col[i], p.n, r[i]);
          continue;
        }
        if (L) mx4_fwht<L ? L : 4>(r[i], a);
        const uint32_t b = mx4_scale(mx4_absmax(r[i]), p.ceil);
        const uint32_t code = mx4_codes(r[i], b) ^ (b == 255u ? 0u : flips);
        if (col[i] < p.n) {
          reinterpret_cast<uint32_t*>(p.codes)[(row * p.n + col[i]) >> 3] = code;
          if ((a & 3) == 0) p.scales[(row * p.n + col[i]) >> 5] = (uint8_t)b;
        }
      }
    }
    slot ^= 2;
  }
}

template <int XT, int DT, int WAVES, int CH>
static void launch_n4(const NormArgs& a, hipStream_t s) {
  // 16 waves a compute unit, unless that leaves them uneven numbers of few rows
  const int64_t most = 256 * 16 / WAVES;
  const dim3 grid((unsigned)(a.rows < 4 * most ? a.rows : most)), threads(64 * WAVES);
  if (!a.codes) hipLaunchKernelGGL((norm_kernel<XT, DT, WAVES, CH, false, 0>), grid, threads, 0, s, a);
  else if (a.order == 0) hipLaunchKernelGGL((norm_kernel<XT, DT, WAVES, CH, true, 0>), grid, threads, 0, s, a);
  else if (a.order == 32) hipLaunchKernelGGL((norm_kernel<XT, DT, WAVES, CH, true, 4>), grid, threads, 0, s, a);
  else if (a.order == 64) hipLaunchKernelGGL((norm_kernel<XT, DT, WAVES, CH, true, 8>), grid, threads, 0, s, a);
  else if (a.order == 128) hipLaunchKernelGGL((norm_kernel<XT, DT, WAVES, CH, true, 16>), grid, threads, 0, s, a);
  else hipLaunchKernelGGL((norm_kernel<XT, DT, WAVES, CH, true, 32>), grid, threads, 0, s, a);
}

template <int XT, int DT>
static void launch_n2(const NormArgs& a, hipStream_t s) {
  if (a.n <= 512) launch_n4<XT, DT, 1, 1>(a, s);
  else if (a.n <= 2048) launch_n4<XT, DT, 4, 1>(a, s);
  else if (a.n <= 4096) launch_n4<XT, DT, 8, 1>(a, s);
  else if (a.n <= 8192) launch_n4<XT, DT, 8, 2>(a, s);
  else if (a.n <= 16384) launch_n4<XT, DT, 16, 2>(a, s);
  else launch_n4<XT, DT, 16, 4>(a, s);
}

hipError_t launch_norm(const NormArgs& a, hipStream_t s) {
  if (a.x_dtype == kDtBf16) launch_n2<kDtBf16, kDtBf16>(a, s);
  else if (a.x_dtype == kDtF16) launch_n2<kDtF16, kDtF16>(a, s);
  else if (a.dtype == kDtBf16) launch_n2<kDtF32, kDtBf16>(a, s);
  else if (a.dtype == kDtF16) launch_n2<kDtF32, kDtF16>(a, s);
  else launch_n2<kDtF32, kDtF32>(a, s);
  return hipGetLastError();
}

}  // namespace hr
