// The 4-bit key/value cache: keys and values rotated and quantized as they are
// written, and read back.
//
// What is computed, for the key and the value x of every (token, head), a
// vector of dim elements:
//   y = H_dim (d * x) / sqrt(dim)   (y = x without the rotation)
//   per group: a = max |y|, s = fp16(a / 7), k = 1 / s (0 when s = 0),
//   q = clamp(rint(y k), -7, 7)
// every step one correctly rounded fp32 operation (a / 7 and 1 / s are IEEE
// quotients; y k is rounded before rint).  With the rotation 1/sqrt(dim) and k
// are one factor and its product is rounded to an integer at once.  A (token,
// head) whose key or value holds a non-finite value, or needs a scale past
// 9352 (7 of them are then past fp16, the type attention multiplies in), is
// stored with zero codes and NaN scales in both, so that whoever reads or
// attends to it gets NaN and nobody else does.
// Reading back: x_hat = d * H_dim (q s) / sqrt(dim), rounded once at the end.
//
// A lane holds 8 consecutive elements of its token's key and of its value (one
// 16-byte load each for 16-bit types), so a vector is dim / 8 lanes and a wave
// covers 512 / dim consecutive tokens of one head: their codes are contiguous
// in a page, and so are their scales.  Heads vary fastest over the grid, so
// the workgroups in flight read whole token rows.  Everything stays in
// registers: no LDS.
//
// Bound by memory when there are many tokens: 32768 of 8 heads of 128 in bf16
// (169 MB either way) are written in 39 us, 4.3 TB/s, and read back in 33 us,
// 5.1 TB/s, where a large copy reaches 5.0.  Writing also issues some 400 vector
// instructions for 2 KB of input a wave, a quarter of them the transform; a
// transform on 4-point dot products and nontemporal loads left its time as it
// was.  Bound by the launch when there are few: one token 3.3 and
// 3.0 us, 1237 plain fp32 ones of 8 heads of 64 3.4 and 4.3.
#include "kv4_device.h"

namespace hr {

constexpr int kKv4Threads = 256;
constexpr int kKv4Waves = kKv4Threads / 64;
constexpr float kMaxScale = 9352.0f;     // 7 of these are an fp16 number

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

// What a lane's 16 bytes of K and of V come to: codes and group scale.
template <int D, bool ROT>
__device__ __forceinline__ void quantize_pair(float* w, int a, int group, int lane, uint32_t* code, _Float16* s16,
                                              bool* bad_out) {
#pragma clang fp contract(off)
  constexpr int L = D / 8;
  if (ROT) fwht_lanes2<L>(w, a);
  // group scales; a non-finite input makes every rotated value non-finite, so
  // the absmax sees it; without the rotation x * 0 does
  bool bad = false;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const float* x = w + 8 * kv;
    float m = fabsf(x[0]), z = 0.0f;
#pragma unroll
    for (int e = 1; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));
    if (!ROT) {
#pragma unroll
      for (int e = 0; e < 8; ++e) z = x[e] * 0.0f + z;
    }
    const float am = __uint_as_float(group_max(__float_as_uint(m), group));
    float s32 = div7(ROT ? am * kv4_norm<D>() : am);
    asm("" : "+v"(s32));       // rounded to fp32 before fp16: a mixed-precision fma would round once
    s16[kv] = (_Float16)s32;
    bad |= !((float)s16[kv] <= kMaxScale) || z != z;
  }
  const uint64_t bads = __builtin_amdgcn_ballot_w64(bad);
  const uint64_t mine = (L == 64 ? ~0ull : (1ull << L) - 1) << (lane & ~(L - 1));
  bad = (bads & mine) != 0;
  *bad_out = bad;
  // a code passes 7 only against a scale rounded down in fp16's subnormals
  const bool clamp = __builtin_amdgcn_ballot_w64(fminf((float)s16[0], (float)s16[1]) < 6.103515625e-05f) != 0;
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
      if (ROT) {
        r[e] = fmaf(w[8 * kv + e], k, M);
      } else {
        const float y = w[8 * kv + e] * k;
        r[e] = y + M;
      }
    }
    if (clamp) {
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] = __builtin_amdgcn_fmed3f(r[e], M - 7.0f, M + 7.0f);
    }
    code[kv] = bad ? 0u : pack8(r);
  }
}

// SETS groups of 512 / D tokens a wave, all loads first.
template <int D, int DT, bool ROT, int SETS>
__global__ __launch_bounds__(kKv4Threads) void kv4_append_kernel(Kv4AppendArgs p) {
  constexpr int L = D / 8, VPW = 64 / L;
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int tb = blockIdx.x / p.c.heads, head = blockIdx.x - tb * p.c.heads;
  const int64_t t0 = ((int64_t)tb * kKv4Waves + wave) * (VPW * SETS) + lane / L;
  const int a = ROT ? kv4_logical<L>(lane) : lane & (L - 1);
  float w[SETS][16];
  int64_t slot[SETS];
#pragma unroll
  for (int u = 0; u < SETS; ++u) {
    // past the end: the last token again, written nowhere
    const int64_t t = t0 + u * VPW < p.tokens ? t0 + u * VPW : p.tokens - 1;
    slot[u] = p.slots[t];
    if (t0 + u * VPW >= p.tokens) slot[u] = -1;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const int64_t at = t * p.stride[kv] + head * D + 8 * a;
      if (DT == kDtF32) load_vec<DT, 8>(reinterpret_cast<const float*>(p.x[kv]) + at, w[u] + 8 * kv);
      else load_vec<DT, 8>(reinterpret_cast<const uint16_t*>(p.x[kv]) + at, w[u] + 8 * kv);
    }
  }
  uint32_t sg[8];
  if (ROT) load_signs<8>(p.c.signs, 8 * a, sg);
  const int gl = p.c.group >> 3;                       // lanes of a group
#pragma unroll
  for (int u = 0; u < SETS; ++u) {
    if (ROT) {
#pragma unroll
      for (int e = 0; e < 16; ++e) w[u][e] = flip(w[u][e], sg[e & 7]);
    }
    uint32_t code[2];
    _Float16 s16[2];
    bool bad;
    quantize_pair<D, ROT>(w[u], a, p.c.group, lane, code, s16, &bad);
    const int64_t page_id = slot[u] >> p.c.page_log2;
    if (slot[u] < 0 || page_id >= p.c.pages) continue;
    const int off = (int)slot[u] & ((1 << p.c.page_log2) - 1);
    const int64_t block = page_id * p.c.heads + head;
    const int64_t cat = ((block << p.c.page_log2) + off) * (D / 8) + a;
    const int64_t sat = ((block * (D / p.c.group) + a / gl) << p.c.page_log2) + off;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      reinterpret_cast<uint32_t*>(p.c.codes[kv])[cat] = code[kv];
      if ((a & (gl - 1)) == 0) p.c.scales[kv][sat] = bad ? __builtin_bit_cast(_Float16, (uint16_t)0x7E00) : s16[kv];
    }
  }
}

template <int D, int DT, bool ROT, int SETS, bool NT>
__global__ __launch_bounds__(kKv4Threads) void kv4_read_kernel(Kv4ReadArgs p) {
  constexpr int L = D / 8, VPW = 64 / L;
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int tb = blockIdx.x / p.c.heads, head = blockIdx.x - tb * p.c.heads;
  const int64_t t0 = ((int64_t)tb * kKv4Waves + wave) * (VPW * SETS) + lane / L;
  const int a = ROT ? kv4_logical<L>(lane) : lane & (L - 1);
  const int ng = D / p.c.group, mine = 8 * a / p.c.group;
  uint32_t x[SETS][2];
  _Float16 s16[SETS][2];
#pragma unroll
  for (int u = 0; u < SETS; ++u) {
    const int64_t t = t0 + u * VPW;
    const int64_t slot = t < p.tokens ? p.slots[t] : -1;
    const int64_t page_id = slot >> p.c.page_log2;
    const int off = (int)slot & ((1 << p.c.page_log2) - 1);
    const int64_t block = page_id * p.c.heads + head;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      x[u][kv] = 0u;
      s16[u][kv] = (_Float16)0;
      if (slot >= 0 && page_id < p.c.pages) {
        x[u][kv] = reinterpret_cast<const uint32_t*>(p.c.codes[kv])[((block << p.c.page_log2) + off) * (D / 8) + a];
        s16[u][kv] = p.c.scales[kv][((block * ng + mine) << p.c.page_log2) + off];
      }
    }
  }
  uint32_t sg[8];
  if (ROT) load_signs<8>(p.c.signs, 8 * a, sg);
  const float f = kv4_norm<D>() * kv4_tau(a);
#pragma unroll
  for (int u = 0; u < SETS; ++u) {
    const int64_t t = t0 + u * VPW;
    float w[16];
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const float s = (float)s16[u][kv];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[8 * kv + e] = (float)(((int)(x[u][kv] << (28 - 4 * e))) >> 28) * s;
    }
    if (ROT) {
      fwht_lanes2<L>(w, a);
#pragma unroll
      for (int e = 0; e < 16; ++e) w[e] = flip(w[e] * f, sg[e & 7]);
    }
    if (t < p.tokens) {
      const int64_t at = (t * p.c.heads + head) * D + 8 * a;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        if (DT == kDtF32) store_vec<DT, 8, NT>(reinterpret_cast<float*>(p.y[kv]) + at, w + 8 * kv);
        else store_vec<DT, 8, NT>(reinterpret_cast<uint16_t*>(p.y[kv]) + at, w + 8 * kv);
      }
    }
  }
}

template <int D>
static unsigned kv4_blocks(int64_t tokens, int heads, int sets) {
  const int64_t per = kKv4Waves * (512 / D) * sets;
  return (unsigned)((tokens + per - 1) / per * heads);
}

// Two sets a wave once that leaves eight waves a SIMD's worth of work: what a
// wave does besides the vectors is then shared.
template <int D>
static int kv4_sets(int64_t tokens, int heads) {
  return kv4_blocks<D>(tokens, heads, 2) >= 2048 ? 2 : 1;
}

template <int D, int DT, bool ROT>
static void append3(const Kv4AppendArgs& a, hipStream_t s) {
  const int sets = kv4_sets<D>(a.tokens, a.c.heads);
  const dim3 g(kv4_blocks<D>(a.tokens, a.c.heads, sets)), b(kKv4Threads);
  if (sets == 2) hipLaunchKernelGGL((kv4_append_kernel<D, DT, ROT, 2>), g, b, 0, s, a);
  else hipLaunchKernelGGL((kv4_append_kernel<D, DT, ROT, 1>), g, b, 0, s, a);
}

// Outputs past half of the L2s' 32 MiB are stored around them.  Appending and
// reading back, two calls: 32768 tokens of 8 heads of 128 in bf16 76 us against
// 81, 4099 of 4 heads of 256 in fp16 16.7 against 18.2.
constexpr int64_t kReadStreamBytes = int64_t(16) << 20;

template <int D, int DT, bool ROT>
static void read3(const Kv4ReadArgs& a, hipStream_t s) {
  const int sets = kv4_sets<D>(a.tokens, a.c.heads);
  const dim3 g(kv4_blocks<D>(a.tokens, a.c.heads, sets)), b(kKv4Threads);
  const bool nt = 2 * a.tokens * a.c.heads * D * (DT == kDtF32 ? 4 : 2) >= kReadStreamBytes;
  // two sets a wave are 32 MiB of outputs or more
  if (sets == 2) hipLaunchKernelGGL((kv4_read_kernel<D, DT, ROT, 2, true>), g, b, 0, s, a);
  else if (nt) hipLaunchKernelGGL((kv4_read_kernel<D, DT, ROT, 1, true>), g, b, 0, s, a);
  else hipLaunchKernelGGL((kv4_read_kernel<D, DT, ROT, 1, false>), g, b, 0, s, a);
}

template <int D, int DT>
static void append2(const Kv4AppendArgs& a, hipStream_t s) {
  if (a.c.rotate) append3<D, DT, true>(a, s);
  else append3<D, DT, false>(a, s);
}

template <int D, int DT>
static void read2(const Kv4ReadArgs& a, hipStream_t s) {
  if (a.c.rotate) read3<D, DT, true>(a, s);
  else read3<D, DT, false>(a, s);
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
