// What the kernels of attention over the 4-bit key/value cache share: which
// tokens a query row sees, matrix instructions, codes to fp16, the last steps
// of an output row.
#pragma once

#include "kv4_device.h"

namespace hr {

constexpr float kLog2e = 1.4426950408889634f;
// Probabilities are fp16 numbers 2^kLift times exp2(score - running maximum): small ones keep their 11 bits down to 2^-25
// of the largest (17 nats below it), which count where the largest belong to tokens of small values.  Scores may pass the
// running maximum by kMaxSlack, in log2 units, before it moves; the two together stay within fp16.  7 and 8 reach 14.6
// nats and cost prompts less (2048 tokens over 8192, 32 heads on 8 of 128: 273 against 275 us, 270 with no lift; 1024 of
// 256 dims 237 against 245), other calls the same.
constexpr float kLift = 11.0f, kMaxSlack = 4.0f;

// The query rows of one sequence, and the tokens they see.  Row and token
// indices fit 32 bits (the host checks); offsets into the cache do not.
// Index arrays do not change during a call: read them through the scalar cache.
__device__ __forceinline__ int read_index(const int32_t* p, int64_t i) {
  return ((const __attribute__((address_space(4))) int32_t*)(uintptr_t)p)[i];
}

struct Kv4Seq {
  int len, s0, news, rows;
  int window, causal;

  __device__ __forceinline__ Kv4Seq(const Kv4AttnArgs& p, int b) : window(p.window), causal(p.causal) {
    const int64_t cap = p.width << p.c.page_log2;
    const int cap32 = cap < kKv4MaxLen ? (int)cap : kKv4MaxLen;
    len = read_index(p.lens, b);
    len = len < 0 ? 0 : len > cap32 ? cap32 : len;
    int s1;
    if (p.starts) {
      s0 = read_index(p.starts, b);
      s1 = read_index(p.starts, b + 1);
    } else {
      s0 = b * p.max_new;
      s1 = s0 + p.max_new;
    }
    if (s0 < 0) s0 = 0;
    if (s1 > (int)p.total) s1 = (int)p.total;
    if (s1 < s0) s1 = s0;        // and s1 - s0 cannot wrap
    news = s1 - s0;
    rows = news * p.rep;
  }
  // new token n sees tokens [lo(n), hi(n)); both grow with n.  In 32 bits: the host keeps windows and lengths to 2^30
  // and new tokens to 2^26.
  __device__ __forceinline__ int lo(int n) const {
    const int v = len - news + n - window + 1;
    return window > 0 && v > 0 ? v : 0;
  }
  __device__ __forceinline__ int hi(int n) const {
    const int v = len - news + n + 1;
    return !causal || v > len ? len : v < 0 ? 0 : v;
  }
};

// The token axis in parts: those of a row tile start at its first visible token
// rounded down to 32, `chunk` tokens each, as many as it takes.
__device__ __forceinline__ int kv4_part_base(int lo) { return lo & ~31; }
__device__ __forceinline__ int kv4_part_count(int lo, int hi, int chunk) {
  const int n = hi - kv4_part_base(lo);
  return n <= 0 ? 1 : (n + chunk - 1) / chunk;
}

__device__ __forceinline__ f32x4 mma(half8v a, half8v b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
// nibbles 0 and 4 (low half, high half) of x as codes in fp16; x's nibbles are two's complement
__device__ __forceinline__ half2v codes_lo(uint32_t x) {
  const half2v h = __builtin_bit_cast(half2v, (x & 0x000F000Fu) ^ 0x64086408u);     // 1024 + 8 + q
  return h - (half2v){(_Float16)1032.0f, (_Float16)1032.0f};
}
// nibbles 1 and 5
__device__ __forceinline__ half2v codes_hi(uint32_t x) {
  const half2v h = __builtin_bit_cast(half2v, (x & 0x00F000F0u) ^ 0x64806480u);     // 1024 + 16 (8 + q)
  const half2v s = {(_Float16)0.0625f, (_Float16)0.0625f}, o = {(_Float16)-72.0f, (_Float16)-72.0f};
  return __builtin_elementwise_fma(h, s, o);
}

// eight codes of a dword in the order nibble 0, 4, 1, 5, 2, 6, 3, 7
__device__ __forceinline__ void codes8(uint32_t x, half2v* h) {
  h[0] = codes_lo(x);
  h[1] = codes_hi(x);
  h[2] = codes_lo(x >> 8);
  h[3] = codes_hi(x >> 8);
}
__device__ constexpr int kOrder[8] = {0, 4, 1, 5, 2, 6, 3, 7};

// byte b (0..3) of x0 and of x1 as two pairs of codes: its low nibbles, its
// high nibbles
__device__ __forceinline__ void codes_of_two(uint32_t x0, uint32_t x1, int b, half2v& lo, half2v& hi) {
  const uint32_t t = __builtin_amdgcn_perm(x1, x0, 0x0c000c00u | (uint32_t)b | ((uint32_t)(4 + b) << 16));
  lo = codes_lo(t);
  hi = codes_hi(t);
}

__device__ __forceinline__ half8v join8(const half2v* h) {
  return (half8v){h[0][0], h[0][1], h[1][0], h[1][1], h[2][0], h[2][1], h[3][0], h[3][1]};
}

// Power of two that brings a row's absmax to [1, 2), as an exponent; 0 for a
// row of zeros or one that is not finite.
__device__ __forceinline__ int row_exponent(float mx) {
  return mx > 0.0f && mx < __builtin_inff() ? __builtin_amdgcn_frexp_expf(mx) - 1 : 0;
}

// An output row's last steps, 16 lanes a row with dims [a D/16, (a + 1) D/16):
// times a weight (1 / the softmax sum), rotated back.
template <int D>
__device__ __forceinline__ void turn_back(int rotate, const int8_t* signs, float weight, int a, float* w) {
  constexpr int NC = D / 16;
  if (!rotate) {
#pragma unroll
    for (int e = 0; e < NC; ++e) w[e] *= weight;
    return;
  }
  fwht_lanes<NC, 16>(w, a);
  const float f = weight * kv4_norm<D>() * kv4_tau(a);
  uint32_t sg[NC];
  load_signs<NC>(signs, a * NC, sg);
#pragma unroll
  for (int e = 0; e < NC; ++e) w[e] = flip(w[e] * f, sg[e]);
}

// The same from the softmax sum; 0 where nothing was seen.
template <int D>
__device__ __forceinline__ void finish_row(int rotate, const int8_t* signs, float l, int a, float* w) {
  turn_back<D>(rotate, signs, l == 0.0f ? 0.0f : 1.0f / l, a, w);
}

}  // namespace hr
