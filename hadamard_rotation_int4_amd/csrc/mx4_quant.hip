// Rows to MXFP4 and back.
//
// What is computed, for every block of 32 consecutive values y of a row (y = x,
// or (I kron H_p)(d * x) / sqrt(p) with Hadamard blocks of order p):
//   a = max |y|,  E = floor(log2 a) - 2 (ceil rule: the smallest E with
//   a <= 6 2^E), at least -127;  scale byte E + 127, 255 when a is not finite
//   code = the e2m1 number nearest to y 2^-E, ties to even, 6 beyond it.
// The scale is a power of two, so without a rotation every step is exact but
// the one rounding to a code.  Reading back is q 2^E, rotated back by
// d * (I kron H_p) / sqrt(p) and rounded once to the output type.
//
// A lane takes an octet of a row (8 elements) and everything stays in
// registers: a Hadamard block is in-lane butterflies and DPP exchanges over
// order / 8 lanes, a scale a maximum over the 4 lanes of a quad.  16-bit rows that
// are rotated go through the matrix cores instead (mx4_rotate.hip).
#include "mx4_device.h"

namespace hr {

constexpr int kMx4Threads = 256;

// Row and octet in it of flat octet o < 2^31, for `per` <= 2^15 octets a row:
// the wave's first octet is divided, the lanes' places behind it take one
// multiplication by magic = floor(2^32 / per) + 1 (exact, as (per + 512) per is
// below 2^32).
struct Mx4Place {
  uint32_t row0, col0, per, magic;
  __device__ __forceinline__ Mx4Place(uint32_t first, uint32_t per_, uint32_t magic_) : per(per_), magic(magic_) {
    row0 = first / per;
    col0 = first - row0 * per;
  }
  __device__ __forceinline__ void at(int offset, int64_t* row, uint32_t* col) const {
    const uint32_t x = col0 + offset, q = __umulhi(x, magic);
    *row = row0 + q;
    *col = x - q * per;
  }
};

static uint32_t mx4_magic(uint32_t per) { return (uint32_t)(((uint64_t)1 << 32) / per + 1); }

template <int DT, int L, int SETS>
__global__ __launch_bounds__(kMx4Threads) void mx4_quant_kernel(Mx4QuantArgs p, int64_t octets, uint32_t magic) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int a = mx4_lane<L>(lane);
  const int64_t first = ((int64_t)blockIdx.x * (kMx4Threads / 64) + wave) * (64 * SETS);
  if (first >= octets) return;
  const Mx4Place place((uint32_t)first, p.n / 8, magic);
  float w[SETS][8];
  uint32_t col[SETS];
#pragma unroll
  for (int u = 0; u < SETS; ++u) {
    int64_t row;
    place.at(64 * u + a, &row, &col[u]);
    if (first + 64 * u + a < octets) {
      load_vec_any<8>(DT, p.x, row * p.x_stride + 8 * col[u], w[u]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[u][e] = 0.0f;
      col[u] = 0;
    }
  }
#pragma unroll
  for (int u = 0; u < SETS; ++u) {
    if (L) {
      uint32_t sg[8];
      load_signs<8>(p.signs, 8 * col[u], sg);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[u][e] = flip(w[u][e], sg[e]);
      mx4_fwht<L>(w[u], a);
      const float f = mx4_negated<L>(a) ? -mx4_norm<L>() : mx4_norm<L>();
#pragma unroll
      for (int e = 0; e < 8; ++e) w[u][e] *= f;
    }
    const uint32_t b = mx4_scale(mx4_absmax(w[u]), p.ceil);
    const uint32_t code = mx4_codes(w[u], b);
    const int64_t o = first + 64 * u + a;
    if (o < octets) {
      reinterpret_cast<uint32_t*>(p.codes)[o] = code;
      if ((a & 3) == 0) p.scales[o >> 2] = (uint8_t)b;
    }
  }
}

template <int DT, int L, int SETS>
__global__ __launch_bounds__(kMx4Threads) void mx4_dequant_kernel(Mx4DequantArgs p, int64_t octets, uint32_t magic) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int a = mx4_lane<L>(lane);
  const int64_t first = ((int64_t)blockIdx.x * (kMx4Threads / 64) + wave) * (64 * SETS);
  if (first >= octets) return;
  uint32_t r[SETS], b[SETS];
#pragma unroll
  for (int u = 0; u < SETS; ++u) {
    const int64_t o = first + 64 * u + a;
    r[u] = 0u;
    b[u] = 0u;
    if (o < octets) {
      r[u] = reinterpret_cast<const uint32_t*>(p.codes)[o];
      b[u] = p.scales[o >> 2];
    }
  }
#pragma unroll
  for (int u = 0; u < SETS; ++u) {
    float w[8];
    mx4_levels(r[u], w);
    const float f = mx4_power(b[u]);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] *= f;
    const int64_t o = first + 64 * u + a;
    if (L) {
      mx4_fwht<L>(w, a);
      const float g = mx4_negated<L>(a) ? -mx4_norm<L>() : mx4_norm<L>();
      uint32_t sg[8];
      int64_t row;
      uint32_t col;
      Mx4Place((uint32_t)first, p.n / 8, magic).at(64 * u + a, &row, &col);
      load_signs<8>(p.signs, o < octets ? 8 * col : 0, sg);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = flip(w[e] * g, sg[e]);
    }
    if (o < octets) store_vec_any<8>(DT, p.y, 8 * o, w);
  }
}

template <int DT, int L>
static void launch_q(const Mx4QuantArgs& a, int64_t octets, hipStream_t s) {
  const int64_t per = kMx4Threads;
  hipLaunchKernelGGL((mx4_quant_kernel<DT, L, 1>), dim3((unsigned)((octets + per - 1) / per)), dim3(kMx4Threads), 0, s, a,
                     octets, mx4_magic(a.n / 8));
}

template <int DT, int L>
static void launch_d(const Mx4DequantArgs& a, int64_t octets, hipStream_t s) {
  const int64_t per = kMx4Threads;
  hipLaunchKernelGGL((mx4_dequant_kernel<DT, L, 1>), dim3((unsigned)((octets + per - 1) / per)), dim3(kMx4Threads), 0, s, a,
                     octets, mx4_magic(a.n / 8));
}

#define HR_MX4_TYPE(launch, a, octets, s)                  \
  do {                                                     \
    if (a.dtype == kDtBf16) launch<kDtBf16, 0>(a, octets, s);  \
    else if (a.dtype == kDtF16) launch<kDtF16, 0>(a, octets, s); \
    else launch<kDtF32, 0>(a, octets, s);                  \
  } while (0)
#define HR_MX4_ORDER(launch, DT, a, octets, s)          \
  switch (a.order) {                                    \
    case 32: launch<DT, 4>(a, octets, s); break;        \
    case 64: launch<DT, 8>(a, octets, s); break;        \
    case 128: launch<DT, 16>(a, octets, s); break;      \
    default: launch<DT, 32>(a, octets, s); break;       \
  }

hipError_t launch_mx4_quant(const Mx4QuantArgs& args, hipStream_t s) {
  Mx4QuantArgs a = args;
  a.stream = a.rows * a.n * (a.dtype == kDtF32 ? 4 : 2) >= kStreamBytes;
  const int64_t octets = a.rows * (a.n / 8);
  if (a.order && a.dtype != kDtF32) launch_mx4_rotate_quant(a, s);
  else if (a.order) HR_MX4_ORDER(launch_q, kDtF32, a, octets, s)
  else HR_MX4_TYPE(launch_q, a, octets, s);
  return hipGetLastError();
}

hipError_t launch_mx4_dequant(const Mx4DequantArgs& args, hipStream_t s) {
  Mx4DequantArgs a = args;
  a.stream = a.rows * a.n * (a.dtype == kDtF32 ? 4 : 2) >= kStreamBytes;
  const int64_t octets = a.rows * (a.n / 8);
  if (a.order && a.dtype != kDtF32) launch_mx4_rotate_back(a, s);
  else if (a.order) HR_MX4_ORDER(launch_d, kDtF32, a, octets, s)
  else HR_MX4_TYPE(launch_d, a, octets, s);
  return hipGetLastError();
}

}  // namespace hr
