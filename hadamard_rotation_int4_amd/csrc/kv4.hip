// The 4-bit key/value cache: keys and values rotated and quantized as they are
// written, and read back.
//
// What is computed, for the key and the value x of every (token, head), a
// vector of dim elements:
//   y = H_dim (d * x) / sqrt(dim)   (y = x without the rotation)
//   per group: a = max |y|, s = fp16(a / 7), k = 1 / s (0 when s = 0),
//   q = clamp(rint(y k), -7, 7)
// every step one correctly rounded fp32 operation (a / 7 and 1 / s are IEEE
// quotients; y k is rounded before rint; with the rotation, 1/sqrt(dim) and k
// are one factor).  A (token, head) whose key or value holds a non-finite
// value, or needs a scale above the fp16 range, is stored with zero codes and
// NaN scales in both, so that whoever reads or attends to it gets NaN and
// nobody else does.
// Reading back: x_hat = d * H_dim (q s) / sqrt(dim), rounded once at the end.
//
// A lane holds 8 consecutive elements of its token's key and of its value (one
// 16-byte load each for 16-bit types), so a vector is dim / 8 lanes and a wave
// covers 512 / dim consecutive tokens of one head: their codes are contiguous
// in a page, and so are their scales.  Heads vary fastest over the grid, so
// the workgroups in flight read whole token rows.  Everything stays in
// registers: no LDS.  Bound by memory when there are many tokens and by the
// launch when there are few.
#include "kv4_device.h"

namespace hr {

constexpr int kKv4Threads = 256;
constexpr int kKv4Waves = kKv4Threads / 64;

// Group absmax over the group's lanes (non-negative floats and NaN compare as
// integers, NaN above all).
__device__ __forceinline__ uint32_t group_max(uint32_t a, int group) {
  a = umax_dpp<kQuadXor1>(a);
  a = umax_dpp<kQuadXor2>(a);
  if (group >= 64) a = umax_dpp<kRowHalfMirror>(a);
  if (group >= 128) a = umax_dpp<kRowMirror>(a);
  if (group >= 256) {
    const auto sw = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    a = sw[0] > sw[1] ? sw[0] : sw[1];
  }
  return a;
}

template <int D, int DT, bool ROT>
__global__ __launch_bounds__(kKv4Threads) void kv4_append_kernel(Kv4AppendArgs p) {
#pragma clang fp contract(off)
  constexpr int L = D / 8, VPW = 64 / L;
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int head = blockIdx.x % p.c.heads;
  const int64_t t = ((int64_t)(blockIdx.x / p.c.heads) * kKv4Waves + wave) * VPW + lane / L;
  const int a = ROT ? kv4_logical<L>(lane) : lane & (L - 1);
  const bool in = t < p.tokens;
  const int64_t slot = in ? p.slots[t] : -1;
  float w[2][8];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    if (in) {
      const int64_t at = t * p.stride[kv] + head * D + 8 * a;
      if (DT == kDtF32) load_vec<DT, 8>(reinterpret_cast<const float*>(p.x[kv]) + at, w[kv]);
      else load_vec<DT, 8>(reinterpret_cast<const uint16_t*>(p.x[kv]) + at, w[kv]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[kv][e] = 0.0f;
    }
  }
  if (ROT) {
    uint32_t sg[8];
    load_signs<8>(p.c.signs, 8 * a, sg);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[kv][e] = flip(w[kv][e], sg[e]);
      fwht_lanes<8, L>(w[kv], a);
    }
  }
  // group scales; a non-finite input makes every rotated value non-finite, so
  // the absmax sees it; without the rotation x * 0 does
  _Float16 s16[2];
  bool bad = false;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    float m = fabsf(w[kv][0]), z = 0.0f;
#pragma unroll
    for (int e = 1; e < 8; ++e) m = fmaxf(m, fabsf(w[kv][e]));
    if (!ROT) {
#pragma unroll
      for (int e = 0; e < 8; ++e) z = w[kv][e] * 0.0f + z;
    }
    const float am = __uint_as_float(group_max(__float_as_uint(m), p.c.group));
    float s32 = div7(ROT ? am * kv4_norm<D>() : am);
    asm("" : "+v"(s32));       // rounded to fp32 before fp16: a mixed-precision fma would round once
    s16[kv] = (_Float16)s32;
    bad |= !((float)s16[kv] < __builtin_inff()) || z != z;
  }
  const uint64_t bads = __builtin_amdgcn_ballot_w64(bad);
  const uint64_t mine = (L == 64 ? ~0ull : (1ull << L) - 1) << (lane & ~(L - 1));
  bad = (bads & mine) != 0;
  const int64_t page_id = slot >> p.c.page_log2;
  if (slot < 0 || page_id >= p.c.pages) return;
  const int off = (int)(slot & ((1 << p.c.page_log2) - 1));
  const int64_t block = page_id * p.c.heads + head;
  const int gl = p.c.group >> 3;                       // lanes of a group
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const float s = (float)s16[kv];
    float k = s > 0.0f ? 1.0f / s : 0.0f;
    if (ROT) k *= kv4_norm<D>() * kv4_tau(a);
    // the sum with 1.5 * 2^23 + 8 holds q + 8 in its low bits (ties to even)
    constexpr float M = 12582920.0f;
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float y = w[kv][e] * k;
      r[e] = __builtin_amdgcn_fmed3f(y + M, M - 7.0f, M + 7.0f);
    }
    const uint32_t code = bad ? 0u : pack8(r);
    reinterpret_cast<uint32_t*>(p.c.codes[kv])[(((block << p.c.page_log2) + off) * D >> 3) + a] = code;
    if ((a & (gl - 1)) == 0) {
      const int64_t at = ((block * (D / p.c.group) + a / gl) << p.c.page_log2) + off;
      p.c.scales[kv][at] = bad ? __builtin_bit_cast(_Float16, (uint16_t)0x7E00) : s16[kv];
    }
  }
}

template <int D, int DT, bool ROT>
__global__ __launch_bounds__(kKv4Threads) void kv4_read_kernel(Kv4ReadArgs p) {
  constexpr int L = D / 8, VPW = 64 / L;
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int head = blockIdx.x % p.c.heads;
  const int64_t t = ((int64_t)(blockIdx.x / p.c.heads) * kKv4Waves + wave) * VPW + lane / L;
  const int a = ROT ? kv4_logical<L>(lane) : lane & (L - 1);
  const bool in = t < p.tokens;
  const int64_t slot = in ? p.slots[t] : -1;
  const int64_t page_id = slot >> p.c.page_log2;
  const bool live = slot >= 0 && page_id < p.c.pages;
  const int off = (int)(slot & ((1 << p.c.page_log2) - 1));
  const int64_t block = page_id * p.c.heads + head;
  uint32_t x[2] = {0u, 0u};
  float s[2] = {0.0f, 0.0f};
  if (live) {
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      x[kv] = reinterpret_cast<const uint32_t*>(p.c.codes[kv])[(((block << p.c.page_log2) + off) * D >> 3) + a];
      s[kv] = (float)p.c.scales[kv][((block * (D / p.c.group) + 8 * a / p.c.group) << p.c.page_log2) + off];
    }
  }
  uint32_t sg[8];
  if (ROT) load_signs<8>(p.c.signs, 8 * a, sg);
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = (float)(((int)(x[kv] << (28 - 4 * e))) >> 28) * s[kv];
    if (ROT) {
      fwht_lanes<8, L>(w, a);
      const float f = kv4_norm<D>() * kv4_tau(a);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = flip(w[e] * f, sg[e]);
    }
    if (in) {
      const int64_t at = (t * p.c.heads + head) * D + 8 * a;
      if (DT == kDtF32) store_vec<DT, 8>(reinterpret_cast<float*>(p.y[kv]) + at, w);
      else store_vec<DT, 8>(reinterpret_cast<uint16_t*>(p.y[kv]) + at, w);
    }
  }
}

template <int D>
static unsigned kv4_blocks(int64_t tokens, int heads) {
  const int64_t per = kKv4Waves * (512 / D);
  return (unsigned)((tokens + per - 1) / per * heads);
}

template <int D, int DT>
static void append2(const Kv4AppendArgs& a, hipStream_t s) {
  const dim3 g(kv4_blocks<D>(a.tokens, a.c.heads)), b(kKv4Threads);
  if (a.c.rotate) hipLaunchKernelGGL((kv4_append_kernel<D, DT, true>), g, b, 0, s, a);
  else hipLaunchKernelGGL((kv4_append_kernel<D, DT, false>), g, b, 0, s, a);
}

template <int D, int DT>
static void read2(const Kv4ReadArgs& a, hipStream_t s) {
  const dim3 g(kv4_blocks<D>(a.tokens, a.c.heads)), b(kKv4Threads);
  if (a.c.rotate) hipLaunchKernelGGL((kv4_read_kernel<D, DT, true>), g, b, 0, s, a);
  else hipLaunchKernelGGL((kv4_read_kernel<D, DT, false>), g, b, 0, s, a);
}

template <int D>
static void append1(const Kv4AppendArgs& a, hipStream_t s) {
  if (a.dtype == kDtBf16) append2<D, kDtBf16>(a, s);
  else if (a.dtype == kDtF16) append2<D, kDtF16>(a, s);
  else append2<D, kDtF32>(a, s);
}

template <int D>
static void read1(const Kv4ReadArgs& a, hipStream_t s) {
  if (a.dtype == kDtBf16) read2<D, kDtBf16>(a, s);
  else if (a.dtype == kDtF16) read2<D, kDtF16>(a, s);
  else read2<D, kDtF32>(a, s);
}

hipError_t launch_kv4_append(const Kv4AppendArgs& a, hipStream_t s) {
  switch (a.c.dim) {
    case 64: append1<64>(a, s); break;
    case 128: append1<128>(a, s); break;
    default: append1<256>(a, s); break;
  }
  return hipGetLastError();
}

hipError_t launch_kv4_read(const Kv4ReadArgs& a, hipStream_t s) {
  switch (a.c.dim) {
    case 64: read1<64>(a, s); break;
    case 128: read1<128>(a, s); break;
    default: read1<256>(a, s); break;
  }
  return hipGetLastError();
}

}  // namespace hr
