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
// turn, so that every operand is read once.
#include "mx4_device.h"

namespace hr {

// 8 elements of type DT from element `at` of base, which need not be aligned;
// zeros from the n-th of the row on.
template <int DT>
__device__ __forceinline__ void load_octet(const void* base, int64_t at, int col, int n, float* w) {
  if (col + 8 <= n) {
    if (DT == kDtF32) {
      struct __attribute__((packed, aligned(4))) U { float v[8]; };
      const U u = *reinterpret_cast<const U*>(reinterpret_cast<const float*>(base) + at);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = u.v[e];
    } else {
      struct __attribute__((packed, aligned(2))) U { uint32_t v[4]; };
      const U u = *reinterpret_cast<const U*>(reinterpret_cast<const uint16_t*>(base) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (DT == kDtBf16) {
          w[2 * i] = __uint_as_float(u.v[i] << 16);
          w[2 * i + 1] = __uint_as_float(u.v[i] & 0xFFFF0000u);
        } else {
          const half2v h = __builtin_bit_cast(half2v, u.v[i]);
          w[2 * i] = (float)h[0];
          w[2 * i + 1] = (float)h[1];
        }
      }
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    w[e] = 0.0f;
    if (col + e < n) {
      if (DT == kDtF32) w[e] = reinterpret_cast<const float*>(base)[at + e];
      else if (DT == kDtBf16) w[e] = bf16_bits_to_float(reinterpret_cast<const uint16_t*>(base)[at + e]);
      else w[e] = (float)reinterpret_cast<const _Float16*>(base)[at + e];
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

// Sum over the workgroup, the same in every thread; `slot` alternates between
// two calls that no barrier separates.
template <int WAVES>
__device__ __forceinline__ float block_sum(float v, float (*red)[WAVES], int slot) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  if (WAVES == 1) return v;
  if ((threadIdx.x & 63) == 0) red[slot][threadIdx.x >> 6] = v;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) t += red[slot][w];
  return t;
}

// XT, DT: types of the stream and of the block and the norm; CH octets a lane;
// L = 0: no rotation, QUANT: h goes to MXFP4.
template <int XT, int DT, int WAVES, int CH, bool QUANT, int L>
__global__ __launch_bounds__(64 * WAVES) void norm_kernel(NormArgs p) {
  __shared__ float red[2][WAVES];
  // the same labels with and without a rotation, so that sums have one order and
  // r the same bits
  const int a = mx4_lane<16>(threadIdx.x & 63) | (threadIdx.x & ~63);
  const int64_t row = blockIdx.x;
  float r[CH][8];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int col = 8 * (a + i * 64 * WAVES);
    load_octet<XT>(p.x, row * p.x_stride + col, col, p.n, r[i]);
  }
  if (p.block) {
    float u[CH][8];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int col = 8 * (a + i * 64 * WAVES);
      load_octet<DT>(p.block, row * p.block_stride + col, col, p.n, u[i]);
    }
    float f = p.scale;
    if (p.post_norm) {
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum = fmaf(u[i][e], u[i][e], sum);
      f = p.scale / sqrtf(block_sum<WAVES>(sum, red, 0) / (float)p.n + p.eps);
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int col = 8 * (a + i * 64 * WAVES);
      float v[8];
      if (p.post_weight) {
        load_octet<kDtF32>(p.post_weight, col, col, p.n, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[i][e] *= v[e];
      }
      if (p.gate) {
        load_octet<DT>(p.gate, row / p.gate_rows * p.n + col, col, p.n, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) u[i][e] *= v[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) r[i][e] = fmaf(u[i][e], f, r[i][e]);
      if (p.residual) store_octet<XT>(p.residual, row * p.residual_stride + col, col, p.n, r[i]);
    }
  }
  if (!QUANT && !p.h) return;
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(r[i][e], r[i][e], sum);
  const float f = 1.0f / sqrtf(block_sum<WAVES>(sum, red, 1) / (float)p.n + p.eps);
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int col = 8 * (a + i * 64 * WAVES);
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[i][e] *= f;
    if (p.weight) {
      load_octet<kDtF32>(p.weight, col, col, p.n, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) r[i][e] *= v[e];
    }
    if (!QUANT) {
      store_octet<DT>(p.h, row * p.n + col, col, p.n, r[i]);
      continue;
    }
    if (L) {
      uint32_t sg[8];
      load_signs<8>(p.signs, col < p.n ? col : 0, sg);
#pragma unroll
      for (int e = 0; e < 8; ++e) r[i][e] = flip(r[i][e], sg[e]);
      mx4_fwht<L>(r[i], a);
      const float g = mx4_factor<L>(a);
#pragma unroll
      for (int e = 0; e < 8; ++e) r[i][e] *= g;
    }
    const uint32_t b = mx4_scale(mx4_absmax(r[i]), p.ceil);
    const uint32_t code = mx4_codes(r[i], b);
    if (col < p.n) {
      reinterpret_cast<uint32_t*>(p.codes)[(row * p.n + col) >> 3] = code;
      if ((a & 3) == 0) p.scales[(row * p.n + col) >> 5] = (uint8_t)b;
    }
  }
}

template <int XT, int DT, int WAVES, int CH>
static void launch_n4(const NormArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.rows), threads(64 * WAVES);
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
  else if (a.n <= 4096) launch_n4<XT, DT, 4, 2>(a, s);
  else if (a.n <= 16384) launch_n4<XT, DT, 8, 4>(a, s);
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
