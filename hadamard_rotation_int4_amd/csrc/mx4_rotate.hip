// MXFP4 rows of 16-bit types through a Hadamard rotation, to the format and back,
// with the order-32 factor of the transform on the matrix cores.
//
// What is computed: mx4_quant.hip.  H_p = H_{p/32} kron H_32, so the transform of a
// row is H_32 on each of its blocks of 32 and then H_{p/32} across p / 32 consecutive
// blocks.  A wave takes 32 consecutive blocks as the columns of a 32 x 32 product
// with H_32, whose entries are +-1 and products exact: two
// v_mfma_f32_32x32x16.  The other factor is log2(p/32) exchanges between
// neighbouring lanes (columns), one v_fmac_f32_dpp an element; its signs, as in
// kv4_device.h, are one for all of a lane's elements.
//
// Lane (column c, half h) supplies elements 16 h .. 16 h + 15 of its block.  The rows
// of H_32 are given to the instruction in the order in which its results come out
// (v = 0 .. 15 of half h), so that a lane gets back elements 16 h + v: 8 bytes of codes.
//
// Bound by memory: bf16 65536 x 2048, order 128, takes 57 us to the format and 60 back,
// each over and over (339 MB, 5.9 and 5.7 TB/s, where a large copy reaches 5.3 and one
// operand negated 6.1); in turn 79 and 61, the rows read back still on their way to memory
// when the next call's are asked for.  With butterflies on the vector units, 17
// instructions an element, it was their issue (there and back 190 us); this takes 6.
#include "mx4_device.h"

namespace hr {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// (the second launch bound keeps results of matrix instructions out of the
// accumulation registers, from which each would have to be moved)
constexpr int kMxRotThreads = 256;

// H_32's fragments of this lane: rows in result order, columns in operand order.
template <int DT>
__device__ __forceinline__ void hadamard_operand(int lane, u32x4 (&f)[2]) {
  const int i = lane & 31, h = lane >> 5;
  const int out = 16 * ((i >> 2) & 1) + 4 * (i >> 3) + (i & 3);
  constexpr uint32_t ONE = DT == kDtBf16 ? 0x3F80u : 0x3C00u;
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int at = 16 * h + 8 * k + 2 * e;
      const uint32_t lo = ONE | ((__popc(out & at) & 1) << 15), hi = ONE | ((__popc(out & (at + 1)) & 1) << 15);
      f[k][e] = lo | (hi << 16);
    }
}

template <int DT>
__device__ __forceinline__ f32x16 times_hadamard(const u32x4 (&hf)[2], const u32x4 (&x)[2]) {
  f32x16 d = {};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if constexpr (DT == kDtBf16)
      d = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, hf[k]), __builtin_bit_cast(bf16x8, x[k]), d, 0,
                                                  0, 0);
    else
      d = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8v, hf[k]), __builtin_bit_cast(half8v, x[k]), d, 0, 0,
                                                 0);
  }
  return d;
}

// H_{2^S} across the lanes of a column's group, up to the lane's sign; w must not
// come from a matrix instruction directly (the exchanges are inline assembly).
template <int S>
__device__ __forceinline__ void across(float* w, int c) {
  if (S >= 1) {
    const float b = (c & 1) ? -1.0f : 1.0f;
    HR_FMAC_DPP16(w, b, "quad_perm:[1,0,3,2]");
  }
  if (S >= 2) {
    const float b = (c & 2) ? -1.0f : 1.0f;
    HR_FMAC_DPP16(w, b, "quad_perm:[2,3,0,1]");
  }
  if (S >= 3) {
    const float b = (c & 4) ? -1.0f : 1.0f;
    HR_FMAC_DPP16(w, b, "row_half_mirror");
  }
}

// Sign bits of 16 consecutive entries of the diagonal, two to a word as 16-bit
// values lie; `all` flips every one.
__device__ __forceinline__ void sign_words(const int8_t* signs, int first, uint32_t all, uint32_t (&m)[8]) {
  const u32x4 b = signs ? *reinterpret_cast<const u32x4*>(signs + first) : (u32x4){0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // bytes 0, 1 and 2, 3 to the high bytes of two halves
    m[2 * i] = (__builtin_amdgcn_perm(b[i], b[i], 0x010c000cu) & 0x80008000u) ^ all;
    m[2 * i + 1] = (__builtin_amdgcn_perm(b[i], b[i], 0x030c020cu) & 0x80008000u) ^ all;
  }
}

// Where the tiles of a wave lie, in halves of 16 blocks: half g of tile u, of which
// this lane sees block j = c % 16.  ROWS: rows are whole numbers of tiles, and a wave
// takes the same columns of R consecutive rows, one set of signs for all; else tiles
// follow one another over the ends of rows.
template <int R, bool ROWS>
struct MxTiles {
  int64_t rows;
  uint32_t per, magic, group, ct, first, row0, col0, j;
  __device__ __forceinline__ MxTiles(int64_t wave, int j_, int64_t rows_, uint32_t per_, uint32_t magic_)
      : rows(rows_), per(per_), magic(magic_), j(j_) {
    const uint32_t tiles = per / 32;
    group = ROWS ? (uint32_t)wave / tiles : 0;
    ct = (uint32_t)wave - group * tiles;
    first = (uint32_t)wave * 32 * R;
    row0 = ROWS ? 0 : first / per;
    col0 = first - row0 * per;
  }
  // row, first element in it and flat block; past the end the first row again and
  // block -1, stored nowhere
  __device__ __forceinline__ void at(int u, int g, int64_t* row, uint32_t* col, int64_t* block) const {
    if (ROWS) {
      *row = (int64_t)group * R + u;
      *col = 32 * (32 * ct + 16 * g + j);
      *block = *row * per + 32 * ct + 16 * g + j;
    } else {
      const uint32_t x = col0 + 32 * u + 16 * g + j, q = per == 1 ? x : __umulhi(x, magic);
      *row = (int64_t)row0 + q;
      *col = 32 * (x - q * per);
      *block = (int64_t)first + 32 * u + 16 * g + j;
    }
    if (*row >= rows) {
      *row = 0;
      *block = -1;
      if (!ROWS) *col = 0;
    }
  }
};

// Memory's order and the product's.  Lane (c, h) needs both 16-byte quarters 2 h and
// 2 h + 1 of its block, but an instruction that takes quarter 2 h of every block
// would touch half of each line.  Instead instruction g takes the 16 blocks of half
// g whole, rows of lanes with c < 16 their quarters 2 h, the others 2 h + 1, and an
// exchange between rows makes the one of the other (its own inverse).
__device__ __forceinline__ void swap_quarters(u32x4 (&x)[2]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const auto s = __builtin_amdgcn_permlane16_swap(x[0][e], x[1][e], false, false);
    x[0][e] = s[0];
    x[1][e] = s[1];
  }
}

template <int DT, int S, int R, bool ROWS>
__global__ __launch_bounds__(kMxRotThreads, 2) void mx4_rotate_quant_kernel(Mx4QuantArgs p, int64_t waves, uint32_t magic) {
  const int lane = threadIdx.x & 63, c = kv4_logical<32>(lane), h = lane >> 5, g = c >> 4;
  const int64_t wave = (int64_t)blockIdx.x * (kMxRotThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (wave >= waves) return;
  const MxTiles<R, ROWS> tiles(wave, c & 15, p.rows, p.n / 32, magic);
  u32x4 x[R][2];
#pragma unroll
  for (int u = 0; u < R; ++u)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      int64_t row, block;
      uint32_t col;
      tiles.at(u, k, &row, &col, &block);
      const u32x4* src =
          reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(p.x) + row * p.x_stride + col + 8 * (2 * h + g));
      x[u][k] = p.stream ? __builtin_nontemporal_load(src) : *src;
    }
  u32x4 hf[2];
  hadamard_operand<DT>(lane, hf);
  constexpr float NORM = mx4_norm<4 << S>();
  const uint32_t flips = (__popc(c & ((1 << S) - 1)) & 1) ? 0x88888888u : 0u;
  uint32_t m[8];
  f32x16 d[R];
#pragma unroll
  for (int u = 0; u < R; ++u) {
    if (u == 0 || !ROWS) {
      int64_t row, block;
      uint32_t col;
      tiles.at(u, g, &row, &col, &block);
      sign_words(p.signs, col + 16 * h, 0u, m);
    }
    swap_quarters(x[u]);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) x[u][k][e] ^= m[4 * k + e];
    d[u] = times_hadamard<DT>(hf, x[u]);
  }
#pragma unroll
  for (int u = 0; u < R; ++u) {
    float w[16];
#pragma unroll
    for (int v = 0; v < 16; ++v) w[v] = d[u][v] * NORM;
    across<S>(w, c);
    float a = __builtin_elementwise_maximum(mx4_absmax(w), mx4_absmax(w + 8));
    const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(a), false, false);
    const uint32_t b = mx4_scale_byte(sw[0] > sw[1] ? sw[0] : sw[1], p.ceil);
    const uint2 code = make_uint2(mx4_codes(w, b), mx4_codes(w + 8, b));
    int64_t row, block;
    uint32_t col;
    tiles.at(u, g, &row, &col, &block);
    if (block >= 0) {
      const uint32_t f = b == 255u ? 0u : flips;
      *reinterpret_cast<uint2*>(p.codes + block * 16 + 8 * h) = make_uint2(code.x ^ f, code.y ^ f);
      if (h == 0) p.scales[block] = (uint8_t)b;
    }
  }
}

template <int DT, int S, int R, bool ROWS>
__global__ __launch_bounds__(kMxRotThreads, 2) void mx4_rotate_back_kernel(Mx4DequantArgs p, int64_t waves, uint32_t magic) {
  const int lane = threadIdx.x & 63, c = kv4_logical<32>(lane), h = lane >> 5, g = c >> 4;
  const int64_t wave = (int64_t)blockIdx.x * (kMxRotThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (wave >= waves) return;
  const MxTiles<R, ROWS> tiles(wave, c & 15, p.rows, p.n / 32, magic);
  uint2 code[R];
  uint32_t b[R];
#pragma unroll
  for (int u = 0; u < R; ++u) {
    int64_t row, block;
    uint32_t col;
    tiles.at(u, g, &row, &col, &block);
    const int64_t f = block < 0 ? 0 : block;
    code[u] = *reinterpret_cast<const uint2*>(p.codes + f * 16 + 8 * h);
    b[u] = p.scales[f];
  }
  u32x4 hf[2];
  hadamard_operand<DT>(lane, hf);
  constexpr float NORM = mx4_norm<4 << S>();
  const uint32_t flips = (__popc(c & ((1 << S) - 1)) & 1) ? 0x80008000u : 0u;
  uint32_t m[8];
  f32x16 d[R];
#pragma unroll
  for (int u = 0; u < R; ++u) {
    u32x4 x[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) mx4_levels16<DT>(k ? code[u].y : code[u].x, x[k]);
    d[u] = times_hadamard<DT>(hf, x);
  }
#pragma unroll
  for (int u = 0; u < R; ++u) {
    const float f = mx4_power(b[u]) * NORM;
    float w[16];
#pragma unroll
    for (int v = 0; v < 16; ++v) w[v] = d[u][v] * f;
    across<S>(w, c);
    if (u == 0 || !ROWS) {
      int64_t row, block;
      uint32_t col;
      tiles.at(u, g, &row, &col, &block);
      sign_words(p.signs, col + 16 * h, flips, m);
    }
    u32x4 y[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float lo = w[8 * k + 2 * e], hi = w[8 * k + 2 * e + 1];
        if constexpr (DT == kDtBf16) y[k][e] = __builtin_bit_cast(uint32_t, (bf16x2){(__bf16)lo, (__bf16)hi});
        else y[k][e] = __builtin_bit_cast(uint32_t, (half2v){(_Float16)lo, (_Float16)hi});
        y[k][e] ^= m[4 * k + e];
      }
    swap_quarters(y);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      int64_t row, block;
      uint32_t col;
      tiles.at(u, k, &row, &col, &block);
      if (block < 0) continue;
      u32x4* dst = reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(p.y) + block * 32 + 8 * (2 * h + g));
      if (p.stream) __builtin_nontemporal_store(y[k], dst);
      else *dst = y[k];
    }
  }
}

// Tiles of a wave on the way back: two when there are waves enough for every compute
// unit (65536 x 2048, order 128: 60 us, with one 66, with four 65).  On the way there one
// is best (57, 60, 62).
constexpr int64_t kMxManyTiles = 4 * 4096;

template <template <int, int, int, bool> class K, int DT, int S, int MANY, typename Args>
static void launch_rotate(const Args& a, hipStream_t s) {
  const uint32_t per = a.n / 32;
  const int64_t tiles = (a.rows * per + 31) / 32;
  const uint32_t magic = (uint32_t)(((uint64_t)1 << 32) / per + 1);
  auto go = [&](auto kernel, int64_t waves) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)((waves + kMxRotThreads / 64 - 1) / (kMxRotThreads / 64))), dim3(kMxRotThreads),
                       0, s, a, waves, magic);
  };
  if (per % 32) go(K<DT, S, 1, false>::kernel, tiles);
  else if (MANY == 1 || tiles < kMxManyTiles) go(K<DT, S, 1, true>::kernel, tiles);
  else go(K<DT, S, MANY, true>::kernel, (a.rows + MANY - 1) / MANY * (per / 32));
}

template <int DT, int S, int R, bool ROWS>
struct MxTo {
  static constexpr int many = 1;
  static constexpr auto kernel = mx4_rotate_quant_kernel<DT, S, R, ROWS>;
};
template <int DT, int S, int R, bool ROWS>
struct MxBack {
  static constexpr int many = 2;
  static constexpr auto kernel = mx4_rotate_back_kernel<DT, S, R, ROWS>;
};

template <template <int, int, int, bool> class K, int DT, typename Args>
static void launch_order(const Args& a, hipStream_t s) {
  switch (a.order) {
    case 32: launch_rotate<K, DT, 0, K<DT, 0, 1, true>::many>(a, s); break;
    case 64: launch_rotate<K, DT, 1, K<DT, 0, 1, true>::many>(a, s); break;
    case 128: launch_rotate<K, DT, 2, K<DT, 0, 1, true>::many>(a, s); break;
    default: launch_rotate<K, DT, 3, K<DT, 0, 1, true>::many>(a, s); break;
  }
}

void launch_mx4_rotate_quant(const Mx4QuantArgs& a, hipStream_t s) {
  if (a.dtype == kDtBf16) launch_order<MxTo, kDtBf16>(a, s);
  else launch_order<MxTo, kDtF16>(a, s);
}

void launch_mx4_rotate_back(const Mx4DequantArgs& a, hipStream_t s) {
  if (a.dtype == kDtBf16) launch_order<MxBack, kDtBf16>(a, s);
  else launch_order<MxBack, kDtF16>(a, s);
}

}  // namespace hr
