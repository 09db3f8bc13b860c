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
// Everything stays in registers: a Hadamard block is in-lane butterflies and DPP
// exchanges, a scale a maximum over the lanes of a block.  16-bit rows that are
// rotated go through the matrix cores instead (mx4_rotate.hip).
//
// Bound by memory when there are many rows: without a rotation bf16 65536 x 2048 takes
// 57 us to the format and 57 back, each over and over (339 MB, 5.9 TB/s, where a large
// copy reaches 5.3 and one operand negated 6.1), fp32 1237 x 5120 6.8 and 6.9.  fp32 rows
// through a rotation of order 128, operands past the caches: 65536 x 2048 113 us to the format
// and 172 back (608 MB, 5.4 and 3.5 TB/s; back, a lane's two stores are 32 bytes apart),
// 1237 x 5120 8.4 and 11.1.  Bound by the launch when there are few: one row of 4096 1.8 us.
#include "mx4_device.h"

namespace hr {

constexpr int kMx4Threads = 256;
// Chunks a lane without a rotation: two cover the latency better than one and leave more
// waves than four (bf16 65536 x 2048 57, 58 and 60 us; back 57, 64 and 61).
constexpr int kMx4Sets = 2;

// Row and chunk in it of flat chunk o < 2^32, for `per` chunks a row: the wave's first
// chunk is divided, the lanes' places behind it (fewer than 256) are in that row or
// the next where rows are longer than that, and else take one multiplication by
// magic = floor(2^32 / per) + 1, which is exact below 2^32 / per.
struct Mx4Place {
  uint32_t row0, col0, per, magic;
  __device__ __forceinline__ Mx4Place(uint32_t first, uint32_t per_, uint32_t magic_) : per(per_), magic(magic_) {
    row0 = first / per;
    col0 = first - row0 * per;
  }
  __device__ __forceinline__ void at(int offset, int64_t* row, uint32_t* col) const {
    const uint32_t x = col0 + offset, q = per >= 256 ? (x >= per ? 1u : 0u) : __umulhi(x, magic);
    *row = row0 + q;
    *col = x - q * per;
  }
};

static uint32_t mx4_magic(uint32_t per) { return (uint32_t)(((uint64_t)1 << 32) / per + 1); }

// Without a rotation a lane takes 16 bytes of its row, E = 8 or 4 elements, so that
// an instruction reads whole lines; a block is 32 / E lanes.  FLAT: rows follow one
// another.
template <int E>
__device__ __forceinline__ float chunk_absmax(const float* w) {
  float m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(fabsf(w[0]), fabsf(w[1])), fabsf(w[2]));
  m = __builtin_elementwise_maximum(m, fabsf(w[3]));
  if (E == 8) {
    m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, fabsf(w[4])), fabsf(w[5]));
    m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, fabsf(w[6])), fabsf(w[7]));
  }
  return m;
}

template <int DT, bool FLAT, int SETS>
__global__ __launch_bounds__(kMx4Threads) void mx4_plain_quant_kernel(Mx4QuantArgs p, int64_t chunks, uint32_t magic) {
  constexpr int E = DT == kDtF32 ? 4 : 8;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t first = ((int64_t)blockIdx.x * (kMx4Threads / 64) + wave) * (64 * SETS);
  if (first >= chunks) return;
  u32x4 x[SETS];
#pragma unroll
  for (int u = 0; u < SETS; ++u) {
    const int64_t o = first + 64 * u + lane < chunks ? first + 64 * u + lane : chunks - 1;    // the last again
    int64_t at = o * E;
    if (!FLAT) {
      int64_t row;
      uint32_t col;
      Mx4Place((uint32_t)first, p.n / E, magic).at((int)(o - first), &row, &col);
      at = row * p.x_stride + E * col;
    }
    const u32x4* src = reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(p.x) + at * (16 / E));
    x[u] = p.stream ? __builtin_nontemporal_load(src) : *src;
  }
#pragma unroll
  for (int u = 0; u < SETS; ++u) {
    float w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == kDtF32) {
        w[i] = __uint_as_float(x[u][i]);
      } else if constexpr (DT == kDtBf16) {
        w[2 * i] = __uint_as_float(x[u][i] << 16);
        w[2 * i + 1] = __uint_as_float(x[u][i] & 0xFFFF0000u);
      } else {
        const uint32_t v = x[u][i];      // (a bit cast of a vector's element itself takes the first one)
        const half2v h = __builtin_bit_cast(half2v, v);
        w[2 * i] = (float)h[0];
        w[2 * i + 1] = (float)h[1];
      }
    }
    uint32_t a = __float_as_uint(chunk_absmax<E>(w)) & 0x7FFFFFFFu;
    a = umax_dpp<kQuadXor1>(a);
    a = umax_dpp<kQuadXor2>(a);
    if (E == 4) a = umax_dpp<kRowHalfMirror>(a);
    const uint32_t b = mx4_scale_byte(a, p.ceil);
    const int64_t o = first + 64 * u + lane;
    if (o < chunks) {
      if constexpr (E == 8) {
        reinterpret_cast<uint32_t*>(p.codes)[o] = mx4_codes(w, b);
      } else {
        const float s = __uint_as_float(b << 23);
        uint32_t r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, w[0], w[1], s, 0);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, w[2], w[3], s, 1);
        reinterpret_cast<uint16_t*>(p.codes)[o] = (uint16_t)(b == 255u ? 0u : r);
      }
      if ((lane & (32 / E - 1)) == 0) p.scales[o / (32 / E)] = (uint8_t)b;
    }
  }
}

template <int DT, int SETS>
__global__ __launch_bounds__(kMx4Threads) void mx4_plain_back_kernel(Mx4DequantArgs p, int64_t chunks) {
  constexpr int E = DT == kDtF32 ? 4 : 8;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t first = ((int64_t)blockIdx.x * (kMx4Threads / 64) + wave) * (64 * SETS);
  if (first >= chunks) return;
  uint32_t r[SETS], b[SETS];
#pragma unroll
  for (int u = 0; u < SETS; ++u) {
    const int64_t o = first + 64 * u + lane < chunks ? first + 64 * u + lane : chunks - 1;
    r[u] = E == 8 ? reinterpret_cast<const uint32_t*>(p.codes)[o] : reinterpret_cast<const uint16_t*>(p.codes)[o];
    b[u] = p.scales[o / (32 / E)];
  }
#pragma unroll
  for (int u = 0; u < SETS; ++u) {
    float w[8];
    mx4_levels(r[u], w);
    const float f = mx4_power(b[u]);
#pragma unroll
    for (int e = 0; e < E; ++e) w[e] *= f;
    const int64_t o = first + 64 * u + lane;
    if (o < chunks) {
      void* dst = reinterpret_cast<char*>(p.y) + 16 * o;
      if (p.stream) store_vec<DT, E, true>(dst, w);
      else store_vec<DT, E>(dst, w);
    }
  }
}

// fp32 rows with a rotation: a lane takes an octet, 8 elements.
template <int L>
__global__ __launch_bounds__(kMx4Threads) void mx4_quant_kernel(Mx4QuantArgs p, int64_t octets, uint32_t magic) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int a = mx4_lane(lane);
  const int64_t first = ((int64_t)blockIdx.x * (kMx4Threads / 64) + wave) * 64;
  if (first >= octets) return;
  const int64_t o = first + a;
  float w[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  uint32_t col = 0;
  if (o < octets) {
    int64_t row;
    Mx4Place((uint32_t)first, p.n / 8, magic).at(a, &row, &col);
    load_vec<kDtF32, 8>(reinterpret_cast<const float*>(p.x) + row * p.x_stride + 8 * col, w);
  }
  uint32_t sg[8];
  load_signs<8>(p.signs, 8 * col, sg);
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = flip(w[e], sg[e]);
  mx4_fwht(w, a, 8 * L);
  const float f = mx4_negated(a, 8 * L) ? -mx4_norm<L>() : mx4_norm<L>();
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] *= f;
  const uint32_t b = mx4_scale(mx4_absmax(w), p.ceil);
  const uint32_t code = mx4_codes(w, b);
  if (o < octets) {
    reinterpret_cast<uint32_t*>(p.codes)[o] = code;
    if ((a & 3) == 0) p.scales[o >> 2] = (uint8_t)b;
  }
}

template <int L>
__global__ __launch_bounds__(kMx4Threads) void mx4_back_kernel(Mx4DequantArgs p, int64_t octets, uint32_t magic) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int a = mx4_lane(lane);
  const int64_t first = ((int64_t)blockIdx.x * (kMx4Threads / 64) + wave) * 64;
  if (first >= octets) return;
  const int64_t o = first + a;
  uint32_t r = 0u, b = 0u, col = 0;
  if (o < octets) {
    int64_t row;
    Mx4Place((uint32_t)first, p.n / 8, magic).at(a, &row, &col);
    r = reinterpret_cast<const uint32_t*>(p.codes)[o];
    b = p.scales[o >> 2];
  }
  float w[8];
  mx4_levels(r, w);
  const float f = mx4_power(b);
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] *= f;
  mx4_fwht(w, a, 8 * L);
  const float g = mx4_negated(a, 8 * L) ? -mx4_norm<L>() : mx4_norm<L>();
  uint32_t sg[8];
  load_signs<8>(p.signs, 8 * col, sg);
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = flip(w[e] * g, sg[e]);
  if (o < octets) store_vec<kDtF32, 8>(reinterpret_cast<float*>(p.y) + 8 * o, w);
}

template <int L>
static void launch_q(const Mx4QuantArgs& a, hipStream_t s) {
  const int64_t octets = a.rows * (a.n / 8);
  hipLaunchKernelGGL((mx4_quant_kernel<L>), dim3((unsigned)((octets + kMx4Threads - 1) / kMx4Threads)), dim3(kMx4Threads), 0,
                     s, a, octets, mx4_magic(a.n / 8));
}

template <int L>
static void launch_d(const Mx4DequantArgs& a, hipStream_t s) {
  const int64_t octets = a.rows * (a.n / 8);
  hipLaunchKernelGGL((mx4_back_kernel<L>), dim3((unsigned)((octets + kMx4Threads - 1) / kMx4Threads)), dim3(kMx4Threads), 0,
                     s, a, octets, mx4_magic(a.n / 8));
}

template <int DT>
static void launch_plain_q(const Mx4QuantArgs& a, hipStream_t s) {
  constexpr int E = DT == kDtF32 ? 4 : 8, SETS = kMx4Sets;
  const int64_t chunks = a.rows * (a.n / E), per = kMx4Threads * SETS;
  const dim3 grid((unsigned)((chunks + per - 1) / per));
  if (a.x_stride == a.n)
    hipLaunchKernelGGL((mx4_plain_quant_kernel<DT, true, SETS>), grid, dim3(kMx4Threads), 0, s, a, chunks, 0u);
  else
    hipLaunchKernelGGL((mx4_plain_quant_kernel<DT, false, SETS>), grid, dim3(kMx4Threads), 0, s, a, chunks, mx4_magic(a.n / E));
}

template <int DT>
static void launch_plain_d(const Mx4DequantArgs& a, hipStream_t s) {
  constexpr int E = DT == kDtF32 ? 4 : 8, SETS = kMx4Sets;
  const int64_t chunks = a.rows * (a.n / E), per = kMx4Threads * SETS;
  hipLaunchKernelGGL((mx4_plain_back_kernel<DT, SETS>), dim3((unsigned)((chunks + per - 1) / per)), dim3(kMx4Threads), 0, s, a,
                     chunks);
}

hipError_t launch_mx4_quant(const Mx4QuantArgs& args, hipStream_t s) {
  Mx4QuantArgs a = args;
  a.stream = a.rows * a.n * (a.dtype == kDtF32 ? 4 : 2) >= kStreamBytes;
  if (a.order && a.dtype != kDtF32) launch_mx4_rotate_quant(a, s);
  else if (a.order == 32) launch_q<4>(a, s);
  else if (a.order == 64) launch_q<8>(a, s);
  else if (a.order == 128) launch_q<16>(a, s);
  else if (a.order == 256) launch_q<32>(a, s);
  else if (a.dtype == kDtBf16) launch_plain_q<kDtBf16>(a, s);
  else if (a.dtype == kDtF16) launch_plain_q<kDtF16>(a, s);
  else launch_plain_q<kDtF32>(a, s);
  return hipGetLastError();
}

hipError_t launch_mx4_dequant(const Mx4DequantArgs& args, hipStream_t s) {
  Mx4DequantArgs a = args;
  a.stream = a.rows * a.n * (a.dtype == kDtF32 ? 4 : 2) >= kStreamBytes;
  if (a.order && a.dtype != kDtF32) launch_mx4_rotate_back(a, s);
  else if (a.order == 32) launch_d<4>(a, s);
  else if (a.order == 64) launch_d<8>(a, s);
  else if (a.order == 128) launch_d<16>(a, s);
  else if (a.order == 256) launch_d<32>(a, s);
  else if (a.dtype == kDtBf16) launch_plain_d<kDtBf16>(a, s);
  else if (a.dtype == kDtF16) launch_plain_d<kDtF16>(a, s);
  else launch_plain_d<kDtF32>(a, s);
  return hipGetLastError();
}

}  // namespace hr
