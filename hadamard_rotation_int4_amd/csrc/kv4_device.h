// Device helpers shared by the kernels of the 4-bit key/value cache.
//
// A cache holds pages of `page` tokens (a power of two).  Token vectors are
// addressed by (page id, head, place in the page):
//   codes  [pages][heads][page][dim / 2]       packed int4, two's complement
//   scales [pages][heads][dim / group][page]   fp16
// Scales are token-contiguous per group because the attention kernels take a
// group's scales four tokens at a time.
//
// The head rotation is the randomized Hadamard transform of one head,
// y = H_dim (d * x) / sqrt(dim), Sylvester order.  Here a vector of E L
// elements lies over L lanes, E consecutive elements each: the log2 E low
// index bits are register butterflies, the lane bits DPP exchanges.  DPP has
// lane xor 1, 2, 7 (row_half_mirror) and 8 (row_ror:8) but no xor 4, so the
// lanes of a 16-lane row are relabelled: logical index a = (a0, a1, a2, a3)
// sits in physical lane a0 ^ 2 a1 ^ 7 a2 ^ 8 a3, which is a ^ 3 where a2 is
// set and its own inverse.  An exchanged stage computes own + beta * partner
// (beta = -1 where the lane's bit is set), the butterfly up to the lane sign
// tau = (-1)^popcount(a & 15) that the caller folds into its output factor.
#pragma once

#include "hr_device.h"
#include "kv4.h"
#include "fwht2048.h"

namespace hr {

typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef _Float16 half4v __attribute__((ext_vector_type(4)));
typedef _Float16 half8v __attribute__((ext_vector_type(8)));

constexpr int kRowRor8 = 0x128;

// 1 / sqrt(D)
template <int D>
__device__ __forceinline__ constexpr float kv4_norm() {
  return D == 64 ? 0.125f : D == 128 ? 0.08838834764831845f : 0.0625f;
}

// Logical index of this lane among the L lanes of its vector (L = 8, 16, 32).
template <int L>
__device__ __forceinline__ int kv4_logical(int lane) {
  const int p = lane & (L - 1);
  return p ^ (((p >> 2) & 1) * 3);
}

// (-1)^popcount of the DPP-exchanged bits of logical index a.
__device__ __forceinline__ float kv4_tau(int a) { return (__popc(a & 15) & 1) ? -1.0f : 1.0f; }

template <int N>
__device__ __forceinline__ void fwht_regs(float* w) {
#pragma unroll
  for (int h = 1; h < N; h *= 2)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (!(i & h)) bfly(w[i], w[i + h]);
}

// w := tau * (H_{E L} w) over the L lanes; a = kv4_logical<L>(lane).
template <int E, int L>
__device__ __forceinline__ void fwht_lanes(float* w, int a) {
  fwht_regs<E>(w);
  const float b0 = (a & 1) ? -1.0f : 1.0f, b1 = (a & 2) ? -1.0f : 1.0f;
  const float b2 = (a & 4) ? -1.0f : 1.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) w[e] = fmaf(dpp<kQuadXor1>(w[e]), b0, w[e]);
#pragma unroll
  for (int e = 0; e < E; ++e) w[e] = fmaf(dpp<kQuadXor2>(w[e]), b1, w[e]);
#pragma unroll
  for (int e = 0; e < E; ++e) w[e] = fmaf(dpp<kRowHalfMirror>(w[e]), b2, w[e]);
  if (L >= 16) {
    const float b3 = (a & 8) ? -1.0f : 1.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] = fmaf(dpp<kRowRor8>(w[e]), b3, w[e]);
  }
  if (L >= 32) {
    const float b4 = (a & 16) ? -1.0f : 1.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(w[e]), __float_as_uint(w[e]), false, false);
      w[e] = fmaf(__uint_as_float(s[1]), b4, __uint_as_float(s[0]));
    }
  }
}

// The same for two vectors of 8 elements a lane at once, w[0..7] and w[8..15]:
// one instruction an element and exchange.
template <int L>
__device__ __forceinline__ void fwht_lanes2(float* w, int a) {
  fwht_regs<8>(w);
  fwht_regs<8>(w + 8);
  const float b0 = (a & 1) ? -1.0f : 1.0f, b1 = (a & 2) ? -1.0f : 1.0f;
  const float b2 = (a & 4) ? -1.0f : 1.0f;
  HR_FMAC_DPP16(w, b0, "quad_perm:[1,0,3,2]");
  HR_FMAC_DPP16(w, b1, "quad_perm:[2,3,0,1]");
  HR_FMAC_DPP16(w, b2, "row_half_mirror");
  if (L >= 16) {
    const float b3 = (a & 8) ? -1.0f : 1.0f;
    HR_FMAC_DPP16(w, b3, "row_ror:8");
  }
  if (L >= 32) {
    const float b4 = (a & 16) ? -1.0f : 1.0f;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(w[e]), __float_as_uint(w[e]), false, false);
      w[e] = fmaf(__uint_as_float(s[1]), b4, __uint_as_float(s[0]));
    }
  }
}

// N consecutive elements (N * size a multiple of 8 bytes) of type DT to fp32.
template <int DT, int N>
__device__ __forceinline__ void load_vec(const void* p, float* w) {
  if (DT == kDtF32) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const f32x4 r = reinterpret_cast<const f32x4*>(p)[i / 4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[i + e] = r[e];
    }
    return;
  }
  uint32_t u[N / 2];
  if (N % 8 == 0) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      const u32x4 r = reinterpret_cast<const u32x4*>(p)[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) u[4 * i + e] = r[e];
    }
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint2 r = reinterpret_cast<const uint2*>(p)[i];
      u[2 * i] = r.x;
      u[2 * i + 1] = r.y;
    }
  }
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    if (DT == kDtBf16) {
      w[2 * i] = __uint_as_float(u[i] << 16);
      w[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    } else {
      const half2v h = __builtin_bit_cast(half2v, u[i]);
      w[2 * i] = (float)h[0];
      w[2 * i + 1] = (float)h[1];
    }
  }
}

// N consecutive fp32 values rounded to DT (nearest even) and stored; NT: with
// the nontemporal hint (a branch on a run-time flag would be merged without it).
template <int DT, int N, bool NT = false>
__device__ __forceinline__ void store_vec(void* p, const float* w) {
  if (DT == kDtF32) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const f32x4 v = {w[i], w[i + 1], w[i + 2], w[i + 3]};
      f32x4* q = reinterpret_cast<f32x4*>(p) + i / 4;
      if (NT) __builtin_nontemporal_store(v, q);
      else *q = v;
    }
    return;
  }
  uint32_t u[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    if (DT == kDtBf16) {
      const bf16x2 b = {(__bf16)w[2 * i], (__bf16)w[2 * i + 1]};
      u[i] = __builtin_bit_cast(uint32_t, b);
    } else {
      const half2v h = {(_Float16)w[2 * i], (_Float16)w[2 * i + 1]};
      u[i] = __builtin_bit_cast(uint32_t, h);
    }
  }
  if (N % 8 == 0) {
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
      const u32x4 v = {u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]};
      u32x4* q = reinterpret_cast<u32x4*>(p) + i;
      if (NT) __builtin_nontemporal_store(v, q);
      else *q = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) reinterpret_cast<uint2*>(p)[i] = make_uint2(u[2 * i], u[2 * i + 1]);
  }
}

// The runtime-typed forms of the two above.
template <int N>
__device__ __forceinline__ void load_vec_any(int dt, const void* base, int64_t elem, float* w) {
  if (dt == kDtBf16) load_vec<kDtBf16, N>(reinterpret_cast<const uint16_t*>(base) + elem, w);
  else if (dt == kDtF16) load_vec<kDtF16, N>(reinterpret_cast<const uint16_t*>(base) + elem, w);
  else load_vec<kDtF32, N>(reinterpret_cast<const float*>(base) + elem, w);
}
template <int N>
__device__ __forceinline__ void store_vec_any(int dt, void* base, int64_t elem, const float* w) {
  if (dt == kDtBf16) store_vec<kDtBf16, N>(reinterpret_cast<uint16_t*>(base) + elem, w);
  else if (dt == kDtF16) store_vec<kDtF16, N>(reinterpret_cast<uint16_t*>(base) + elem, w);
  else store_vec<kDtF32, N>(reinterpret_cast<float*>(base) + elem, w);
}

// Sign bits (bit 31) of N consecutive entries of the +-1 diagonal; zeros when
// there is none.
template <int N>
__device__ __forceinline__ void load_signs(const int8_t* signs, int first, uint32_t* m) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const uint32_t b = signs ? *reinterpret_cast<const uint32_t*>(signs + first + i) : 0u;
#pragma unroll
    for (int e = 0; e < 4; ++e) m[i + e] = (b << (24 - 8 * e)) & 0x80000000u;
  }
}
__device__ __forceinline__ float flip(float v, uint32_t m) { return __uint_as_float(__float_as_uint(v) ^ m); }

}  // namespace hr
