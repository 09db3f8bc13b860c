// Attention over the 4-bit key/value cache for many query rows (prompts and
// chunks of prompts), 16-bit queries.  The mathematics is kv4_attention.hip's;
// here it is the matrix products that count, so a workgroup shares each tile's
// codes-to-fp16 work among 128 query rows through LDS.
//
// One workgroup of 4 waves takes 128 query rows of one (sequence, key/value
// head), row = new token * rep + head of the group, and walks over 64-token
// tiles.  Each wave owns 32 rows and computes, on 32x32x16 instructions,
//   S^T = K q'^T (rows: tokens),   O^T = V^T P^T (rows: dims):
// S^T leaves query row n = lane % 32 in the lane, with tokens
// 8 (r / 4) + 4 h + r % 4 in register r (h = lane / 32), which is what the
// second product wants as its right operand when its contraction slots
// (h, i) stand for tokens 8 (i / 4) + 4 h + i % 4.  So probabilities never
// leave their lane, and the softmax needs one exchange (between the two halves
// of a wave), and that only when the running maximum moves.
//
// LDS holds scaled fp16, in 16-byte pieces that a wave reads contiguously:
//   keys    [dim / 8][64 tokens] pieces of 8 dims (in nibble order; the
//           queries are laid out to match), one piece of padding a row so that
//           the four rows a wave writes at once fall into different banks;
//   values  [8 octets][dim] pieces of 8 tokens, octet 2 t + h holding the
//           tokens of slots (h, .) of 16-token step t; a piece's place among
//           the dims is the transposed (dim % (dim/16), dim / (dim/16)), so
//           that 16 lanes that hold neighbouring dims write contiguously.
// Two buffers: while the products read one tile, the next one's codes are on
// their way to registers, and then to the other buffer; one barrier a tile.
//
// Heads vary fastest over the grid, so that with 8 heads the workgroups of one
// head share an XCD's L2; the last rows, which see most, go first.
#include "kv4_attention.h"

namespace hr {

constexpr int kPromptThreads = 256;
constexpr int kPromptWaves = kPromptThreads / 64;
constexpr int kPromptTokens = 64;           // of a tile

typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16 mma32(half8v a, half8v b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// One thread's share of a tile's codes and scales on their way to LDS: a
// quarter of one token's key, and dim / 16 dims of four tokens' values.
template <int D>
struct Share {
  static constexpr int NK = D / 32;                     // key dwords
  static constexpr int NV = (D + 127) / 128;            // value dwords a token
  static constexpr int NS = D == 256 ? 2 : 1;           // 32-dim spans of the key's share with scales of their own
  uint32_t k[NK];
  uint32_t v[4][NV];
  _Float16 ks[NS];
  half4v vs;
};

// Wave w's share is the tile's 16-token block w: one page.
template <int D>
__device__ __forceinline__ void load_share(const Kv4Cache& c, const int32_t* table_row, int head, int j, int last,
                                           int lane, Share<D>& x) {
  if (j > last) j = last & ~15;        // past the end: any block of the sequence, masked
  const int sh = c.page_log2;
  int64_t id = table_row[j >> sh];
  if (id < 0 || id >= c.pages) id = 0;
  const int off = j & ((1 << sh) - 1);
  const int64_t block = id * c.heads + head;
  const uint8_t* kc = c.codes[0] + ((block << sh) + off) * (D / 2);
  const uint8_t* vc = c.codes[1] + ((block << sh) + off) * (D / 2);
  const int64_t sb = ((block * (D / c.group)) << sh) + off;
  const int kt = lane >> 2, kp = lane & 3;              // key: token of the block, quarter
  const int vq = lane >> 4, va = lane & 15;             // value: token quad of the block, dims
  const uint8_t* kk = kc + kt * (D / 2) + kp * (D / 8);
  if (D == 64) {
    const uint2 r = *reinterpret_cast<const uint2*>(kk);
    x.k[0] = r.x;
    x.k[1] = r.y;
  } else {
#pragma unroll
    for (int n = 0; n < D / 128; ++n) {
      const u32x4 r = reinterpret_cast<const u32x4*>(kk)[n];
#pragma unroll
      for (int e = 0; e < 4; ++e) x.k[4 * n + e] = r[e];
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint8_t* vv = vc + (4 * vq + r) * (D / 2) + va * (D / 32);
    if (D == 64) {
      x.v[r][0] = *reinterpret_cast<const uint16_t*>(vv);
    } else if (D == 128) {
      x.v[r][0] = *reinterpret_cast<const uint32_t*>(vv);
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(vv);
      x.v[r][0] = u.x;
      x.v[r][Share<D>::NV - 1] = u.y;
    }
  }
#pragma unroll
  for (int n = 0; n < Share<D>::NS; ++n) x.ks[n] = c.scales[0][sb + (((kp * (D / 4) + 32 * n) / c.group) << sh) + kt];
  x.vs = *reinterpret_cast<const half4v*>(c.scales[1] + sb + ((va * (D / 16) / c.group) << sh) + 4 * vq);
}

template <int D>
struct PromptLds {
  static constexpr int KROW = kPromptTokens * 16 + 16;  // bytes of a row of key pieces
  static constexpr int KEYS = D / 8 * KROW;
  static constexpr int BUF = KEYS + kPromptTokens / 8 * D * 16;
};

// The share to fp16 and into a buffer.  [lo, to): tokens that some row of the
// tile sees; values of others may be anything and become 0.
template <int D>
__device__ __forceinline__ void store_share(const Share<D>& x, char* buf, int wave, int lane, int j0, int lo, int to) {
  typedef PromptLds<D> L;
  const int kt = lane >> 2, kp = lane & 3;
  const int vq = lane >> 4, va = lane & 15;
#pragma unroll
  for (int n = 0; n < D / 32; ++n) {
    half2v h[4];
    codes8(x.k[n], h);
    const _Float16 s = x.ks[Share<D>::NS == 1 ? 0 : n / 4];
#pragma unroll
    for (int u = 0; u < 4; ++u) h[u] = h[u] * (half2v){s, s};
    *reinterpret_cast<half8v*>(buf + (kp * (D / 32) + n) * L::KROW + (16 * wave + kt) * 16) = join8(h);
  }
  const half4v zero4 = {(_Float16)0, (_Float16)0, (_Float16)0, (_Float16)0};
  half4v vs = __builtin_elementwise_max(x.vs, zero4);   // a poisoned token's NaN is in its score
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int j = j0 + 4 * vq + r;
    if (j < lo || j >= to) vs[r] = (_Float16)0;
  }
  const half2v s01 = {vs[0], vs[1]}, s23 = {vs[2], vs[3]};
  char* vb = buf + L::KEYS + (2 * wave + (vq & 1)) * (D * 16) + (vq >> 1) * 8;
#pragma unroll
  for (int b = 0; b < D / 32; ++b) {
    half2v lo2[2], hi2[2];
    codes_of_two(x.v[0][b >> 2], x.v[1][b >> 2], b & 3, lo2[0], hi2[0]);
    codes_of_two(x.v[2][b >> 2], x.v[3][b >> 2], b & 3, lo2[1], hi2[1]);
    lo2[0] = lo2[0] * s01;
    lo2[1] = lo2[1] * s23;
    hi2[0] = hi2[0] * s01;
    hi2[1] = hi2[1] * s23;
    *reinterpret_cast<half4v*>(vb + (2 * b * 16 + va) * 16) = (half4v){lo2[0][0], lo2[0][1], lo2[1][0], lo2[1][1]};
    *reinterpret_cast<half4v*>(vb + ((2 * b + 1) * 16 + va) * 16) = (half4v){hi2[0][0], hi2[0][1], hi2[1][0], hi2[1][1]};
  }
}

// QT: fp16 terms of a query (2 for fp16 queries, whose output shows the
// rounding of one; 1 for bf16)
template <int D, int QT>
__global__ __launch_bounds__(kPromptThreads, D == 256 ? 1 : 2) void kv4_prompt_kernel(Kv4AttnArgs p) {
  typedef PromptLds<D> L;
  constexpr int NC = D / 16, NB = D / 32;
  constexpr int LD = D + 4;
  static_assert(kPromptWaves * 16 * LD * 4 <= 2 * L::BUF, "the output staging fits the buffers");
  __shared__ __attribute__((aligned(16))) char lds[2 * L::BUF];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5, n = lane & 31;
  const int head = blockIdx.x % p.c.heads;
  int rest = blockIdx.x / p.c.heads;
  const int part = rest % p.nsplit;
  rest /= p.nsplit;
  const int b = rest % p.batch;
  const int tile = p.tiles - 1 - rest / p.batch;
  const Kv4Seq q(p, b);
  const int row0 = tile * kPromptRows;
  if (row0 >= q.rows) return;
  // what the workgroup's rows see
  const int row_end = row0 + kPromptRows < q.rows ? row0 + kPromptRows : q.rows;
  const int lo = q.lo(row0 / p.rep), hi = q.hi((row_end - 1) / p.rep);
  const int parts = kv4_part_count(lo, hi, p.chunk);
  if (part >= parts) return;
  const int from = kv4_part_base(lo) + part * p.chunk;
  int to = from + p.chunk;
  if (to > hi || part == p.nsplit - 1) to = hi;
  // what this wave's rows see; a wave past the rows sees nothing
  const int wrow0 = row0 + 32 * wave;
  const bool any = wrow0 < q.rows;
  const int w_first = any ? wrow0 / p.rep : 0;
  const int w_last = any ? ((wrow0 + 31 < q.rows ? wrow0 + 31 : q.rows - 1) / p.rep) : 0;
  const int w_lo = any ? q.lo(w_first) : 0, w_hi = any ? q.hi(w_last) : 0;
  const int all_lo = q.lo(w_last), all_hi = q.hi(w_first);
  const int row = wrow0 + n;
  const bool valid = row < q.rows;
  const int n_mine = valid ? row / p.rep : w_last;
  const int my_lo = q.lo(n_mine), my_hi = valid ? q.hi(n_mine) : 0;

  // queries: lane (h, n) holds dims 16 c + 8 h + e of row n
  half8v qf[QT][NC];
  float qs = p.scale * kLog2e;
  {
    constexpr int E = D / 2;
    float w[E];
    const int64_t at = (int64_t)(q.s0 + n_mine) * p.q_stride + (head * p.rep + (valid ? row - n_mine * p.rep : 0)) * D;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (valid) load_vec_any<8>(p.dtype, p.q, at + 16 * c + 8 * h, w + 8 * c);
      else
#pragma unroll
        for (int e = 0; e < 8; ++e) w[8 * c + e] = 0.0f;
    }
    if (p.c.rotate) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        uint32_t sg[8];
        load_signs<8>(p.c.signs, 16 * c + 8 * h, sg);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[8 * c + e] = flip(w[8 * c + e], sg[e]);
      }
      fwht_regs<E>(w);
      const float bh = h ? -1.0f : 1.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(w[e]), __float_as_uint(w[e]), false, false);
        w[e] = fmaf(__uint_as_float(s[1]), bh, __uint_as_float(s[0])) * kv4_norm<D>();
      }
    }
    float mx = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) mx = fmaxf(mx, fabsf(w[e]));
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(mx), __float_as_uint(mx), false, false);
    const int ex = row_exponent(fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1])));
    qs = ldexpf(qs, ex);
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float y = ldexpf(w[8 * c + kOrder[e]], -ex);
        qf[0][c][e] = (_Float16)y;
        if (QT == 2) qf[QT - 1][c][e] = (_Float16)(y - (float)qf[0][c][e]);
      }
  }

  f32x16 acc[NB];
#pragma unroll
  for (int db = 0; db < NB; ++db)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[db][r] = 0.0f;
  float m = -__builtin_inff(), l = 0.0f;

  const int32_t* table_row = p.table + (int64_t)b * p.width;
  Share<D> x;
  int cur = 0;
  if (from < to) {
    load_share<D>(p.c, table_row, head, from + 16 * wave, to - 1, lane, x);
    store_share<D>(x, lds, wave, lane, from + 16 * wave, lo, to);
    load_share<D>(p.c, table_row, head, from + kPromptTokens + 16 * wave, to - 1, lane, x);
  }
  __syncthreads();
  for (int t0 = from; t0 < to; t0 += kPromptTokens) {
    const char* buf = lds + cur * L::BUF;
    if (t0 < w_hi && t0 + kPromptTokens > w_lo) {
      // S^T of two 32-token blocks
      f32x16 s[2];
#pragma unroll
      for (int st = 0; st < 2; ++st) {
#pragma unroll
        for (int r = 0; r < 16; ++r) s[st][r] = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const half8v a = *reinterpret_cast<const half8v*>(buf + (2 * c + h) * L::KROW + (32 * st + n) * 16);
          if (QT == 2) s[st] = mma32(a, qf[QT - 1][c], s[st]);
          s[st] = mma32(a, qf[0][c], s[st]);
        }
      }
      const int end = all_hi < to ? all_hi : to;
      if (t0 < all_lo || t0 + kPromptTokens > end) {
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int j = t0 + 32 * st + 8 * (r >> 2) + 4 * h + (r & 3);
            if (j < my_lo || j >= my_hi || j >= to) s[st][r] = -__builtin_inff();
          }
      }
      float mx = s[0][0];
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[st][r]);
      mx *= qs;
      if (__builtin_amdgcn_ballot_w64(mx > m + kMaxSlack)) {
        const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(mx), __float_as_uint(mx), false, false);
        const float mn = fmaxf(m, fmaxf(__uint_as_float(sw[0]), __uint_as_float(sw[1])));
        const float f = mn > m ? exp2f(m - mn) : 1.0f;
        m = mn;
        l *= f;
#pragma unroll
        for (int db = 0; db < NB; ++db) acc[db] *= f;
      }
      const float mu = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          s[st][r] = __builtin_amdgcn_exp2f(fmaf(s[st][r], qs, -mu));
          l += s[st][r];
        }
      // O^T over four 16-token steps
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        half8v ph;
#pragma unroll
        for (int i = 0; i < 8; ++i) ph[i] = (_Float16)s[t >> 1][8 * (t & 1) + i];
#pragma unroll
        for (int db = 0; db < NB; ++db) {
          const half8v a = *reinterpret_cast<const half8v*>(buf + L::KEYS + ((2 * t + h) * D + 32 * db + n) * 16);
          acc[db] = mma32(a, ph, acc[db]);
        }
      }
    }
    // the next tile: registers to the other buffer, the one after it to registers
    const int t1 = t0 + kPromptTokens;
    cur ^= 1;
    if (t1 < to) {
      store_share<D>(x, lds + cur * L::BUF, wave, lane, t1 + 16 * wave, lo, to);
      load_share<D>(p.c, table_row, head, t1 + kPromptTokens + 16 * wave, to - 1, lane, x);
    }
    __syncthreads();
  }
  {
    const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
    l = __uint_as_float(sw[0]) + __uint_as_float(sw[1]);
  }

  // output: 16 rows at a time through the wave's own piece of LDS
  float* o_lds = reinterpret_cast<float*>(lds) + wave * 16 * LD;
  const int la = kv4_logical<16>(lane);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if ((n >> 4) == half) {
#pragma unroll
      for (int db = 0; db < NB; ++db)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int pos = 32 * db + 8 * (r >> 2) + 4 * h + (r & 3);
          o_lds[(n & 15) * LD + (pos & 15) * NC + (pos >> 4)] = acc[db][r];
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int step = 0; step < 4; ++step) {
      const int r16 = 4 * step + (lane >> 4);
      float w[NC];
      load_vec<kDtF32, NC>(o_lds + r16 * LD + la * NC, w);
      const int from_lane = 16 * half + r16;
      const float lr = __shfl(l, from_lane, 64), mr = __shfl(m, from_lane, 64);
      const int r2 = wrow0 + 16 * half + r16;
      const bool store = r2 < q.rows;
      const int n2 = store ? r2 / p.rep : 0;
      const int64_t out_row = (int64_t)(q.s0 + n2) * p.q_heads + head * p.rep + (store ? r2 - n2 * p.rep : 0);
      if (parts > 1 && p.nsplit > 1) {
        if (store) {
          const int64_t at = out_row * p.nsplit + part;
          store_vec<kDtF32, NC>(p.part_o + at * D + la * NC, w);
          if (la == 0) p.part_ml[at] = make_float2(mr, lr);
        }
      } else {
        finish_row<D>(p.c.rotate, p.c.signs, lr, la, w);
        if (store) store_vec_any<NC>(p.dtype, p.out, out_row * D + la * NC, w);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <int D>
static void prompt1(const Kv4AttnArgs& a, hipStream_t s) {
  const dim3 g((unsigned)a.groups), b(kPromptThreads);
  if (a.dtype == kDtF16) hipLaunchKernelGGL((kv4_prompt_kernel<D, 2>), g, b, 0, s, a);
  else hipLaunchKernelGGL((kv4_prompt_kernel<D, 1>), g, b, 0, s, a);
}

void launch_kv4_prompt(const Kv4AttnArgs& a, hipStream_t s) {
  switch (a.c.dim) {
    case 64: prompt1<64>(a, s); break;
    case 128: prompt1<128>(a, s); break;
    default: prompt1<256>(a, s); break;
  }
}

}  // namespace hr
