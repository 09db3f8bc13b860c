// Device helpers of the MXFP4 format: blocks of 32 consecutive elements of a
// row, each an e2m1 code (sign bit over the magnitudes 0, 0.5, 1, 1.5, 2, 3, 4,
// 6), and a scale byte b a block that stands for 2^(b - 127).
//
// A lane holds 8 consecutive elements (an octet), a block is the 4 lanes of a
// quad, and a Hadamard block of `order` elements is L = order / 8 lanes in the
// labelling of kv4_device.h (kv4_logical), which keeps quads together.
#pragma once

#include "kv4_device.h"
#include "mx4.h"

namespace hr {

// Workgroup barrier that leaves the caller's own waits as they are (the compiler
// drains every outstanding memory operation before the barriers that it emits).
__device__ __forceinline__ void mx_barrier() { asm volatile("s_barrier" ::: "memory"); }

// 1 / sqrt(8 L)
template <int L>
__device__ __forceinline__ constexpr float mx4_norm() {
  return L == 4 ? 0.17677669529663687f : L == 8 ? 0.125f : L == 16 ? 0.08838834764831845f : 0.0625f;
}

// This lane's octet among the lanes of its wave.
__device__ __forceinline__ int mx4_lane(int lane) { return (lane & ~31) | kv4_logical<32>(lane); }

// Whether mx4_fwht of this order leaves this lane's values negated (an exchange with a
// multiplier of -1 makes own - partner of partner - own; the last one, of order 256,
// is no such exchange); a: its octet in its block.
__device__ __forceinline__ bool mx4_negated(int a, int order) { return __popc(a & (min(order, 128) / 8 - 1)) & 1; }

// w[i] += dpp(w[i]) * sigma for 8 registers, as HR_FMAC_DPP16.
#define HR_FMAC_DPP8(w, sigma, CTRL) \
  asm volatile("s_nop 1\n\t" \
"v_fmac_f32_dpp %0, %0, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t" \
"v_fmac_f32_dpp %1, %1, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t" \
"v_fmac_f32_dpp %2, %2, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t" \
"v_fmac_f32_dpp %3, %3, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t" \
"v_fmac_f32_dpp %4, %4, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t" \
"v_fmac_f32_dpp %5, %5, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t" \
"v_fmac_f32_dpp %6, %6, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t" \
"v_fmac_f32_dpp %7, %7, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t" \
  : "+v"(w[0]), "+v"(w[1]), "+v"(w[2]), "+v"(w[3]), "+v"(w[4]), "+v"(w[5]), "+v"(w[6]), "+v"(w[7]) \
  : "v"(sigma))

// w[0..7] := H_order w over order / 8 lanes, negated where mx4_negated; a: the lane's
// octet in its block.  Order 0 leaves w as it is.
__device__ __forceinline__ void mx4_fwht(float* w, int a, int order) {
  if (order == 0) return;
  fwht_regs<8>(w);
  const float b0 = (a & 1) ? -1.0f : 1.0f, b1 = (a & 2) ? -1.0f : 1.0f;
  HR_FMAC_DPP8(w, b0, "quad_perm:[1,0,3,2]");
  HR_FMAC_DPP8(w, b1, "quad_perm:[2,3,0,1]");
  if (order >= 64) {
    const float b2 = (a & 4) ? -1.0f : 1.0f;
    HR_FMAC_DPP8(w, b2, "row_half_mirror");
  }
  if (order >= 128) {
    const float b3 = (a & 8) ? -1.0f : 1.0f;
    HR_FMAC_DPP8(w, b3, "row_ror:8");
  }
  if (order >= 256) {
    const float b4 = (a & 16) ? -1.0f : 1.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(w[e]), __float_as_uint(w[e]), false, false);
      w[e] = fmaf(__uint_as_float(s[1]), b4, __uint_as_float(s[0]));
    }
  }
}

// Largest magnitude of 8 elements; NaN if one is.
__device__ __forceinline__ float mx4_absmax(const float* w) {
  float m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(fabsf(w[0]), fabsf(w[1])), fabsf(w[2]));
  m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, fabsf(w[3])), fabsf(w[4]));
  m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, fabsf(w[5])), fabsf(w[6]));
  return __builtin_elementwise_maximum(m, fabsf(w[7]));
}

// Scale byte of a block from the bits of its largest magnitude.  The exponent of
// the largest less that of 4 (the largest binade of e2m1), so that it scales to
// [4, 8) and what is over 6 saturates; with `ceil` one more where it is over 6.  Not
// below 2^-127; 255 when the largest is not finite (infinity and NaN have the
// highest bits, so an integer maximum finds them).
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t a, int ceil) {
  // adding what takes a mantissa over 0.5 past 1 raises the exponent
  const uint32_t e = (a + (ceil ? 0x3FFFFFu : 0u)) >> 23;
  const uint32_t b = e > 2u ? e - 2u : 0u;
  return a >= 0x7F800000u ? 255u : b;
}

// The same for the block of this quad, from the lane's own largest magnitude m.
__device__ __forceinline__ uint32_t mx4_scale(float m, int ceil) {
  uint32_t a = __float_as_uint(m) & 0x7FFFFFFFu;
  a = umax_dpp<kQuadXor1>(a);
  a = umax_dpp<kQuadXor2>(a);
  return mx4_scale_byte(a, ceil);
}

// The 8 codes of w under scale byte b, element e in bits 4 e .. 4 e + 3:
// nearest, ties to even, saturating at 6; 0 under byte 255.
__device__ __forceinline__ uint32_t mx4_codes(const float* w, uint32_t b) {
  const float s = __uint_as_float(b << 23);
  uint32_t r = 0u;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, w[0], w[1], s, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, w[2], w[3], s, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, w[4], w[5], s, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, w[6], w[7], s, 3);
  return b == 255u ? 0u : r;
}

// The 8 magnitudes with signs that codes stand for, before their scale.
__device__ __forceinline__ void mx4_levels(uint32_t r, float* w) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 q0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r, 1.0f, 0);
  const f32x2 q1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r, 1.0f, 1);
  const f32x2 q2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r, 1.0f, 2);
  const f32x2 q3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(r, 1.0f, 3);
  w[0] = q0[0]; w[1] = q0[1]; w[2] = q1[0]; w[3] = q1[1];
  w[4] = q2[0]; w[5] = q2[1]; w[6] = q3[0]; w[7] = q3[1];
}

// The same in 16 bits, two to a word (every level is exact in either type).
template <int DT>
__device__ __forceinline__ void mx4_levels16(uint32_t r, u32x4& x) {
  if constexpr (DT == kDtBf16) {
    x[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r, 1.0f, 0));
    x[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r, 1.0f, 1));
    x[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r, 1.0f, 2));
    x[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r, 1.0f, 3));
  } else {
    x[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(r, 1.0f, 0));
    x[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(r, 1.0f, 1));
    x[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(r, 1.0f, 2));
    x[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(r, 1.0f, 3));
  }
}

// 2^(b - 127): a subnormal for b = 0, NaN for 255.
__device__ __forceinline__ float mx4_power(uint32_t b) {
  return __uint_as_float(b == 0u ? 0x00400000u : b == 255u ? 0x7FC00000u : b << 23);
}

}  // namespace hr
