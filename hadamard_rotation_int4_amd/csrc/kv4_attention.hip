// Attention over the 4-bit key/value cache.
//
// What is computed, for query row (t, h) of sequence b, the i-th of its `new`
// rows, at position pos = len - new + i, key/value head h / rep:
//   q' = H_dim (d * q) / sqrt(dim)            (q' = q without the rotation)
//   z_j = scale q' . (s_j c_j)                over the cached tokens j < len,
//         j <= pos (causal), j > pos - window (window > 0)
//   out = d * H_dim (sum_j softmax(z)_j v_j) / sqrt(dim),  0 for a row that
//         sees no token.
// The rotation is orthogonal, so this is attention over the keys and values
// that the cache stands for, without ever rotating them back.
//
// kv4_attn_kernel.  One workgroup of 4 waves takes 16 query rows of one
// (sequence, key/value head) -- the rep heads that share it times the new
// tokens -- and one part of the token axis; its waves take 32-token tiles in
// turn.  Both products are 16x16x32 matrix instructions in the transposed form
//   S^T = K q'^T  (rows: tokens),    O^T = V^T P^T  (rows: dims),
// which needs no exchange between lanes and no LDS:
// * keys: lane (g, i) = (lane / 16, lane % 16) loads dims [g dim/4, (g+1) dim/4)
//   of token i, dim/8 bytes, and feeds dword c of them to instruction c.  The
//   contraction index is free as long as both operands agree, so the queries
//   are laid out to match, nibble order included.
// * S^T comes out with query row i in the lane and tokens 4 g + r: what the
//   second product wants as its right operand, taken as contraction slots
//   8 g + 4 t + r of the tile's two 16-token blocks t.
// * values: lane (g, i) loads dims [i dim/16, (i+1) dim/16) of those same eight
//   tokens.  Instruction c takes nibble c of each, a byte permute pairing two
//   tokens; its row i is dim i dim/16 + c, so a lane ends up with dim/4
//   consecutive dims of one query row.
// A nibble becomes an fp16 number by planting it in the mantissa of 1024 (or of
// 1024 times a power of two, for the nibble above) and subtracting.
// Scales multiply S (one group a head) or the fp16 keys; values are scaled in
// fp16.  Sums, the running maximum and the softmax sum are fp32; the
// probabilities are rounded to fp16 (2^-12, an eighth of a bf16 output's own
// rounding) and summed as rounded, by a product with ones.
// The running maximum moves only when some score passes it by 2^8, so most
// tiles need neither the exchange between lanes nor the rescale.
//
// fp32 queries: every operand as a sum of bf16 terms (the queries and
// probabilities three, the scaled codes two, which hold them exactly), all
// products above 2^-24 of the whole kept.
//
// Rows of parts are joined by kv4_join_kernel, in the order of the parts.
#include "kv4_attention.h"

namespace hr {

constexpr int kAttnThreads = 256;
constexpr int kAttnWaves = kAttnThreads / 64;

// modes: one group a head / several, 16-bit queries; fp32 queries
enum { kOneGroup = 0, kGroups = 1, kF32 = 2 };

// Waves a SIMD the registers are kept for.  At two or more the compiler takes
// at most 256 registers and leaves the accumulators among the ordinary ones
// (with more it moves them to and from the accumulation registers, 112 moves a
// tile).
constexpr int kv4_attn_waves(int dim, int mode) { return dim == 256 ? (mode == kF32 ? 1 : 2) : mode == kF32 ? 2 : 3; }

// max over the four lanes that hold the same query row (lanes i + 16 g)
__device__ __forceinline__ float max_over_g(float v) {
  auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
  s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}

// x as a sum of bf16 terms
template <int N>
__device__ __forceinline__ void bf16_terms(float x, __bf16* t) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    t[i] = (__bf16)x;
    x -= (float)t[i];
  }
}

// the codes and scales of one 32-token tile, as one lane holds them
template <int D, int MODE>
struct Tile {
  static constexpr int NK = D / 32;                       // key dwords a token
  static constexpr int NB = D / 32;                       // value bytes a token
  static constexpr int NS = MODE == kOneGroup ? 1 : D / 128 > 0 ? D / 128 : 1;   // 32-dim spans with scales of their own
  uint32_t k[2][NK];
  uint32_t v[8][(NB + 3) / 4];
  half4v ks4[2];                                          // one group: tokens 4 g + r
  _Float16 ks1[2][NS];                                    // several: token i, the lane's dims
  half4v vs[2];
};

template <int D, int MODE>
__device__ __forceinline__ void load_tile(const Kv4Cache& c, const int32_t* table_row, int head, int t0,
                                          int last, int g, int i, Tile<D, MODE>& x) {
  const int sh = c.page_log2, pmask = (1 << sh) - 1;
  const int ng = D / c.group;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    // a block past the last token reads that token's block instead (it is masked)
    int j = t0 + 16 * t;
    if (j > last) j = last & ~15;
    int64_t id = table_row[j >> sh];
    if (id < 0 || id >= c.pages) id = 0;
    const int off = j & pmask;
    const int64_t block = id * c.heads + head;
    const uint8_t* kc = c.codes[0] + ((block << sh) + off) * (D / 2);
    const uint8_t* vc = c.codes[1] + ((block << sh) + off) * (D / 2);
    const _Float16* ks = c.scales[0] + ((block * ng) << sh) + off;
    const _Float16* vs = c.scales[1] + ((block * ng) << sh) + off;
    const uint32_t* kp = reinterpret_cast<const uint32_t*>(kc + i * (D / 2) + g * (D / 8));
    if (D == 64) {
      const uint2 r = *reinterpret_cast<const uint2*>(kp);
      x.k[t][0] = r.x;
      x.k[t][1] = r.y;
    } else {
#pragma unroll
      for (int n = 0; n < D / 128; ++n) {
        const u32x4 r = reinterpret_cast<const u32x4*>(kp)[n];
#pragma unroll
        for (int e = 0; e < 4; ++e) x.k[t][4 * n + e] = r[e];
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint8_t* vp = vc + (4 * g + r) * (D / 2) + i * (D / 32);
      if (D == 64) {
        x.v[4 * t + r][0] = *reinterpret_cast<const uint16_t*>(vp);
      } else if (D == 128) {
        x.v[4 * t + r][0] = *reinterpret_cast<const uint32_t*>(vp);
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(vp);
        x.v[4 * t + r][0] = u.x;
        x.v[4 * t + r][D / 256] = u.y;
      }
    }
    if (MODE == kOneGroup) {
      x.ks4[t] = *reinterpret_cast<const half4v*>(ks + 4 * g);
      x.vs[t] = *reinterpret_cast<const half4v*>(vs + 4 * g);
    } else {
#pragma unroll
      for (int n = 0; n < Tile<D, MODE>::NS; ++n) x.ks1[t][n] = ks[(((g * (D / 4) + 32 * n) / c.group) << sh) + i];
      x.vs[t] = *reinterpret_cast<const half4v*>(vs + ((i * (D / 16) / c.group) << sh) + 4 * g);
    }
  }
}

template <int D, int MODE>
__global__ __launch_bounds__(kAttnThreads, kv4_attn_waves(D, MODE)) void kv4_attn_kernel(Kv4AttnArgs p) {
  constexpr int NK = D / 32;             // matrix instructions over the dims
  constexpr int NC = D / 16;             // 16-dim slices of the output
  constexpr int LD = D + 4;              // row pitch of the exchange
  __shared__ float o_lds[kAttnWaves][16][LD];
  __shared__ float m_lds[kAttnWaves][16], l_lds[kAttnWaves][16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, i = lane & 15;
  const int b = blockIdx.y;
  const int head = blockIdx.x % p.c.heads;
  const int rest = blockIdx.x / p.c.heads;
  const int tile = rest % p.tiles, part = rest / p.tiles;

  const Kv4Seq q(p, b);
  const int row0 = tile * 16;
  if (row0 >= q.rows) return;
  // what the tile's first and last row see, and this lane's row
  const int n_first = row0 / p.rep;
  const int n_last = (row0 + 15 < q.rows ? row0 + 15 : q.rows - 1) / p.rep;
  const int lo = q.lo(n_first), hi = q.hi(n_last);
  const int all_lo = q.lo(n_last), all_hi = q.hi(n_first);   // [all_lo, all_hi): seen by every row
  const int row = row0 + i;
  const bool valid = row < q.rows;
  const int n_mine = valid ? row / p.rep : n_last;
  const int my_lo = q.lo(n_mine), my_hi = q.hi(n_mine);
  const int q_row = q.s0 + n_mine;
  const int q_head = head * p.rep + (valid ? row - n_mine * p.rep : 0);
  // this part of the token axis; the last part takes what is left
  const int from = (lo & ~31) + part * p.chunk;
  int to = part == p.nsplit - 1 ? hi : from + p.chunk;
  if (to > hi) to = hi;

  // queries: rotate, scale to [1, 2) by a power of two (kept in qf), lay out as the right operand
  half8v qh[MODE == kF32 ? 1 : NK];
  bf16x8v qb[MODE == kF32 ? NK : 1][3];
  float qf = p.scale * kLog2e;
  {
    constexpr int E = D / 4;
    float w[E];
    if (valid) load_vec_any<E>(p.dtype, p.q, (int64_t)q_row * p.q_stride + q_head * D + g * E, w);
    else
#pragma unroll
      for (int e = 0; e < E; ++e) w[e] = 0.0f;
    if (p.c.rotate) {
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        uint32_t sg[4];
        load_signs<4>(p.c.signs, g * E + e, sg);
#pragma unroll
        for (int u = 0; u < 4; ++u) w[e + u] = flip(w[e + u], sg[u]);
      }
      fwht_regs<E>(w);
      const float b0 = (g & 1) ? -1.0f : 1.0f, b1 = (g & 2) ? -1.0f : 1.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(w[e]), __float_as_uint(w[e]), false, false);
        const float u = fmaf(__uint_as_float(s[1]), b0, __uint_as_float(s[0]));
        s = __builtin_amdgcn_permlane32_swap(__float_as_uint(u), __float_as_uint(u), false, false);
        w[e] = fmaf(__uint_as_float(s[1]), b1, __uint_as_float(s[0])) * kv4_norm<D>();
      }
    }
    if (MODE == kF32) {
#pragma unroll
      for (int c = 0; c < NK; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          __bf16 t[3];
          bf16_terms<3>(w[8 * c + kOrder[e]], t);
#pragma unroll
          for (int u = 0; u < 3; ++u) qb[c][u][e] = t[u];
        }
    } else {
      float mx = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) mx = fmaxf(mx, fabsf(w[e]));
      mx = max_over_g(mx);
      const int ex = row_exponent(mx);
      qf = ldexpf(qf, ex);
#pragma unroll
      for (int c = 0; c < NK; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) qh[c][e] = (_Float16)ldexpf(w[8 * c + kOrder[e]], -ex);
    }
  }

  f32x4 acc[NC], accl = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int c = 0; c < NC; ++c) acc[c] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  float m = -__builtin_inff();
  const half8v ones_h = {(_Float16)1, (_Float16)1, (_Float16)1, (_Float16)1, (_Float16)1, (_Float16)1, (_Float16)1, (_Float16)1};
  const __bf16 one_b = (__bf16)1.0f;
  const bf16x8v ones_b = {one_b, one_b, one_b, one_b, one_b, one_b, one_b, one_b};

  const int32_t* table_row = p.table + (int64_t)b * p.width;
  Tile<D, MODE> x;
  int t0 = from + 32 * wave;
  if (t0 < to) load_tile<D, MODE>(p.c, table_row, head, t0, to - 1, g, i, x);
  for (; t0 < to; t0 += 32 * kAttnWaves) {
    Tile<D, MODE> nx;
    {
      const int t1 = t0 + 32 * kAttnWaves < to ? t0 + 32 * kAttnWaves : t0;
      load_tile<D, MODE>(p.c, table_row, head, t1, to - 1, g, i, nx);
    }
    // S^T
    f32x4 s[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int c = 0; c < NK; ++c) {
        half2v h[4];
        codes8(x.k[t][c], h);
        if (MODE == kOneGroup) {
          s[t] = mma(join8(h), qh[c], s[t]);
        } else {
          const _Float16 sc = x.ks1[t][Tile<D, MODE>::NS == 1 ? 0 : c / 4];
          if (MODE == kGroups) {
#pragma unroll
            for (int u = 0; u < 4; ++u) h[u] = h[u] * (half2v){sc, sc};
            s[t] = mma(join8(h), qh[c], s[t]);
          } else {
            bf16x8v k0, k1;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              __bf16 y[2];
              bf16_terms<2>((float)h[u >> 1][u & 1] * (float)sc, y);
              k0[u] = y[0];
              k1[u] = y[1];
            }
            s[t] = mma(k1, qb[c][1], s[t]);
            s[t] = mma(k0, qb[c][2], s[t]);
            s[t] = mma(k1, qb[c][0], s[t]);
            s[t] = mma(k0, qb[c][1], s[t]);
            s[t] = mma(k0, qb[c][0], s[t]);
          }
        }
      }
    // scores of this lane's row at tokens t0 + 16 t + 4 g + r
    float z[8];
    half4v vs[2];
    const half4v zero4 = {(_Float16)0, (_Float16)0, (_Float16)0, (_Float16)0};
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int r = 0; r < 4; ++r) z[4 * t + r] = MODE == kOneGroup ? s[t][r] * (float)x.ks4[t][r] : s[t][r];
      // a poisoned token has NaN scales: its score carries that to the rows that see it, its value must not
      vs[t] = __builtin_elementwise_max(x.vs[t], zero4);
    }
    if (t0 < all_lo || t0 + 32 > (all_hi < to ? all_hi : to)) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int j = t0 + 16 * (u >> 2) + 4 * g + (u & 3);
        if (j < my_lo || j >= my_hi || j >= to) z[u] = -__builtin_inff();
        if (j < lo || j >= to) vs[u >> 2][u & 3] = (_Float16)0;    // never written: may hold anything
      }
    }
    float mx = z[0];
#pragma unroll
    for (int u = 1; u < 8; ++u) mx = fmaxf(mx, z[u]);
    mx *= qf;
    if (__builtin_amdgcn_ballot_w64(mx > m + kMaxSlack)) {
      const float mn = fmaxf(m, max_over_g(mx));
      const float f = mn > m ? exp2f(m - mn) : 1.0f;
      m = mn;
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[c] *= f;
      accl *= f;
    }
    const float mu = m == -__builtin_inff() ? 0.0f : m;
    float pr[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) pr[u] = __builtin_amdgcn_exp2f(fmaf(z[u], qf, -mu));
    // O^T
    if (MODE != kF32) {
      half8v ph;
#pragma unroll
      for (int u = 0; u < 8; ++u) ph[u] = (_Float16)pr[u];
      accl = mma(ones_h, ph, accl);
#pragma unroll
      for (int bb = 0; bb < NC / 2; ++bb) {
        half2v vl[4], vh[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const half2v sc = {vs[j >> 1][2 * (j & 1)], vs[j >> 1][2 * (j & 1) + 1]};
          codes_of_two(x.v[2 * j][bb >> 2], x.v[2 * j + 1][bb >> 2], bb & 3, vl[j], vh[j]);
          vl[j] = vl[j] * sc;
          vh[j] = vh[j] * sc;
        }
        acc[2 * bb] = mma(join8(vl), ph, acc[2 * bb]);
        acc[2 * bb + 1] = mma(join8(vh), ph, acc[2 * bb + 1]);
      }
    } else {
      bf16x8v pt[3];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        __bf16 t[3];
        bf16_terms<3>(pr[u], t);
#pragma unroll
        for (int e = 0; e < 3; ++e) pt[e][u] = t[e];
      }
#pragma unroll
      for (int e = 2; e >= 0; --e) accl = mma(ones_b, pt[e], accl);
#pragma unroll
      for (int bb = 0; bb < NC / 2; ++bb) {
        bf16x8v v0[2], v1[2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          half2v vv[2];
          codes_of_two(x.v[2 * j][bb >> 2], x.v[2 * j + 1][bb >> 2], bb & 3, vv[0], vv[1]);
#pragma unroll
          for (int d = 0; d < 2; ++d)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              __bf16 y[2];
              bf16_terms<2>((float)vv[d][e] * (float)vs[j >> 1][2 * (j & 1) + e], y);
              v0[d][2 * j + e] = y[0];
              v1[d][2 * j + e] = y[1];
            }
        }
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          f32x4& o = acc[2 * bb + d];
          o = mma(v1[d], pt[1], o);
          o = mma(v0[d], pt[2], o);
          o = mma(v1[d], pt[0], o);
          o = mma(v0[d], pt[1], o);
          o = mma(v0[d], pt[0], o);
        }
      }
    }
    x = nx;
  }

  // join the waves: lane (g, i) holds dims [g D/4, (g+1) D/4) of row i
  if (g == 0) m_lds[wave][i] = m;
  __syncthreads();
  float top = m_lds[0][i];
#pragma unroll
  for (int w = 1; w < kAttnWaves; ++w) top = fmaxf(top, m_lds[w][i]);
  const float f = m == -__builtin_inff() ? 0.0f : exp2f(m - top);
  if (g == 0) l_lds[wave][i] = accl[0] * f;
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < NC; c += 4)
      *reinterpret_cast<f32x4*>(&o_lds[wave][i][(4 * g + r) * NC + c]) =
          (f32x4){acc[c][r] * f, acc[c + 1][r] * f, acc[c + 2][r] * f, acc[c + 3][r] * f};
  __syncthreads();
  // 16 lanes a row, D/16 consecutive dims each
  const int orow = threadIdx.x >> 4;
  const int la = kv4_logical<16>(lane);
  float w[NC], l = 0.0f, mt = m_lds[0][orow];
#pragma unroll
  for (int e = 0; e < NC; ++e) w[e] = 0.0f;
#pragma unroll
  for (int v = 0; v < kAttnWaves; ++v) {
    l += l_lds[v][orow];
    mt = fmaxf(mt, m_lds[v][orow]);
#pragma unroll
    for (int e = 0; e < NC; e += 4) {
      const f32x4 r = *reinterpret_cast<const f32x4*>(&o_lds[v][orow][la * NC + e]);
#pragma unroll
      for (int u = 0; u < 4; ++u) w[e + u] += r[u];
    }
  }
  const int r2 = row0 + orow;
  const bool store = r2 < q.rows;
  const int n2 = store ? r2 / p.rep : 0;
  const int64_t out_row = (int64_t)(q.s0 + n2) * p.q_heads + head * p.rep + (store ? r2 - n2 * p.rep : 0);
  if (p.nsplit > 1) {
    if (store) {
      const int64_t at = out_row * p.nsplit + part;
      store_vec<kDtF32, NC>(p.part_o + at * D + la * NC, w);
      if (la == 0) p.part_ml[at] = make_float2(mt, l);
    }
    return;
  }
  finish_row<D>(p.c, l, la, w);
  if (store) store_vec_any<NC>(p.dtype, p.out, out_row * D + la * NC, w);
}

// One workgroup joins the parts of one output row: its 16 lane groups take the
// parts in turn, LDS adds the groups up, the first group rotates back.
template <int D>
__global__ __launch_bounds__(kAttnThreads) void kv4_join_kernel(Kv4AttnArgs p) {
  constexpr int NC = D / 16;
  __shared__ float o_lds[16][D + 4];
  __shared__ float l_lds[16];
  const int lane = threadIdx.x & 63;
  const int grp = threadIdx.x >> 4;
  const int la = kv4_logical<16>(lane);
  const int b = blockIdx.y;
  const int n = blockIdx.x / p.q_heads;
  const Kv4Seq q(p, b);
  if (n >= q.news) return;
  const int64_t out_row = (int64_t)(q.s0 + n) * p.q_heads + (blockIdx.x - n * p.q_heads);
  const float2* ml = p.part_ml + out_row * p.nsplit;
  float top = -__builtin_inff();
  for (int s = lane; s < p.nsplit; s += 64) top = fmaxf(top, ml[s].x);
  top = wave_max(top);
  float w[NC], l = 0.0f;
#pragma unroll
  for (int e = 0; e < NC; ++e) w[e] = 0.0f;
  for (int s = grp; s < p.nsplit; s += 16) {
    const float2 v = ml[s];
    const float f = v.x == -__builtin_inff() ? 0.0f : exp2f(v.x - top);
    l += v.y * f;
    float o[NC];
    load_vec<kDtF32, NC>(p.part_o + (out_row * p.nsplit + s) * D + la * NC, o);
#pragma unroll
    for (int e = 0; e < NC; ++e) w[e] = fmaf(o[e], f, w[e]);
  }
  store_vec<kDtF32, NC>(&o_lds[grp][la * NC], w);
  if (la == 0) l_lds[grp] = l;
  __syncthreads();
  if (grp >= 4) return;      // the first wave goes on (all of it: the exchanges need whole rows)
#pragma unroll
  for (int e = 0; e < NC; ++e) w[e] = 0.0f;
  l = 0.0f;
  for (int s = 0; s < 16; ++s) {
    l += l_lds[s];
#pragma unroll
    for (int e = 0; e < NC; ++e) w[e] += o_lds[s][la * NC + e];
  }
  finish_row<D>(p.c, l, la, w);
  if (grp == 0) store_vec_any<NC>(p.dtype, p.out, out_row * D + la * NC, w);
}

// Which kernel, and into how many parts of the token axis: enough workgroups to
// fill the chip (three a CU of 16 rows, two of 128), none with fewer than 256
// tokens (two tiles a wave) or, of 128 rows, 512.
void kv4_attention_plan(Kv4AttnArgs* a) {
  const int64_t rows = (int64_t)a->max_new * a->rep;
  a->prompt = a->dtype != kDtF32 && rows > 32;
  const int64_t rows_of = a->prompt ? kPromptRows : 16, least = a->prompt ? 512 : 256;
  const int64_t want = a->prompt ? 512 : 768;
  a->tiles = (int)((rows + rows_of - 1) / rows_of);
  int64_t span = a->max_len;
  if (a->window > 0 && (int64_t)a->window + a->max_new + 31 < span) span = (int64_t)a->window + a->max_new + 31;
  const int64_t groups = (int64_t)a->batch * a->c.heads * a->tiles;
  int64_t n = groups > 0 ? (want + groups - 1) / groups : 1;
  const int64_t most = (span + least - 1) / least;
  if (n > most) n = most;
  if (n < 1) n = 1;
  int64_t chunk = ((span + n - 1) / n + 127) / 128 * 128;
  if (chunk < least) chunk = least;
  n = (span + chunk - 1) / chunk;
  a->nsplit = (int)(n < 1 ? 1 : n);
  a->chunk = (int)chunk;
}

template <int D>
static void attn1(const Kv4AttnArgs& a, hipStream_t s) {
  const dim3 g((unsigned)((int64_t)a.c.heads * a.tiles * a.nsplit), a.batch), b(kAttnThreads);
  if (a.prompt) launch_kv4_prompt(a, s);
  else if (a.dtype == kDtF32) hipLaunchKernelGGL((kv4_attn_kernel<D, kF32>), g, b, 0, s, a);
  else if (a.c.group == D) hipLaunchKernelGGL((kv4_attn_kernel<D, kOneGroup>), g, b, 0, s, a);
  else hipLaunchKernelGGL((kv4_attn_kernel<D, kGroups>), g, b, 0, s, a);
  if (a.nsplit > 1)
    hipLaunchKernelGGL(kv4_join_kernel<D>, dim3((unsigned)(a.max_new * a.q_heads), a.batch), b, 0, s, a);
}

hipError_t launch_kv4_attention(const Kv4AttnArgs& a, hipStream_t s) {
  switch (a.c.dim) {
    case 64: attn1<64>(a, s); break;
    case 128: attn1<128>(a, s); break;
    default: attn1<256>(a, s); break;
  }
  return hipGetLastError();
}

}  // namespace hr
