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
// kv4_attn_kernel.  One workgroup of 4 or 8 waves takes 16 (or 32) query rows of one
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
// probabilities are rounded to fp16 (2^-12 of those down to 2^-25 of the largest,
// an eighth of a bf16 output's own rounding; see kLift) and summed as rounded, by a
// product with ones.
// The running maximum moves only when some score passes it by 2^4, so most
// tiles need neither the exchange between lanes nor the rescale.
//
// fp16 outputs would show the rounding of the queries and keys (4.5e-4 and 4e-4
// rms of an output, where its own is 2.1e-4): for fp16 queries these are two
// fp16 terms each, queries always, keys and values where several groups make a
// scaled code more than 11 bits (two terms hold it exactly).  Probabilities stay
// one term, whose rounding averages out over the tokens: with it outputs are off by
// 2.2e-4 to 2.5e-4.  fp32 queries have the two terms too, and probabilities in two
// terms: all products above 2^-22 of the whole are there.
//
// Single tokens: 64 sequences of 1100 to 8192 tokens, 32 heads on 8 of 128 dims (311
// MB of cache) 75 us, 4.1 TB/s, one of 131071 (138 MB) 29 us, 4.7 TB/s, where a
// large read reaches 5.7.  The first without its arithmetic took 63 to 72 of 74,
// without its loads 44; its parts are cut from the bound on the lengths, and only
// 1.6 waves a SIMD are there on average where three fit.  With several new tokens a
// sequence it is the wait for the chain from a sequence's length over its page
// ids to its codes, in workgroups of few tiles a wave: 12 sequences of up to 6000
// tokens, 5 new ones each, 40 heads on 8, two groups a head, 25 us, where 57% of
// the waves' cycles were waits with 32 rows a workgroup and half the workgroups, and
// 43% are now.
// What was measured and not kept: equal shares of all tokens for every
// workgroup (each then looks for its place first: slower), 8 waves everywhere,
// other orders of the workgroups, deeper prefetch (registers), keys left as
// codes plus an offset taken back by a sum of the queries (1 to 2%).
//
// Rows of parts are joined by kv4_join_kernel, in the order of the parts: 4 to 5
// us, mostly a launch and three loads that wait for each other.
#include "kv4_attention.h"

namespace hr {

constexpr int kFewParts = 8;

// what the fp16 operands have to hold: enough for bf16, fp16 or fp32 outputs
enum { kForBf16 = 0, kForF16 = 1, kForF32 = 2 };

// Waves a SIMD the registers are kept for.  At two or more the compiler takes
// at most 256 registers and leaves the accumulators among the ordinary ones
// (with more it moves them to and from the accumulation registers, 112 moves a
// tile).  Some forms then spill: 50 registers with 128 dims, several groups, fp16, 32
// rows, 2 with bf16 and 16 rows; with 256 dims 20 to 62 with several groups (9 to 11
// fp32), up to 10 with one.
constexpr int kv4_attn_waves(int dim, bool groups, int rows, int prec) {
  return dim == 256 || rows > 16 || (dim == 128 && (prec == kForF32 || (groups && prec == kForF16))) ? 2 : 3;
}

// max over the four lanes that hold the same query row (lanes i + 16 g)
__device__ __forceinline__ float max_over_g(float v) {
  auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
  s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}

// the codes and scales of one 32-token tile, as one lane holds them
template <int D, bool GROUPS>
struct Tile {
  static constexpr int NK = D / 32;                       // key dwords a token
  static constexpr int NB = D / 32;                       // value bytes a token
  static constexpr int NS = GROUPS && D == 256 ? 2 : 1;   // 32-dim spans with scales of their own
  uint32_t k[2][NK];
  uint32_t v[8][(NB + 3) / 4];
  half4v ks4[2];                                          // one group: tokens 4 g + r
  half2v ks1[NS];                                         // several: token i of both blocks, the lane's dims
  half4v vs[2];
};

// Where the tokens of a tile are, the page ids one tile ahead of the codes.
struct Ids {
  int id[2];
};
__device__ __forceinline__ Ids load_ids(const Kv4Cache& c, const int32_t* table_row, int t0, int last) {
  // past the last token, that token's tile instead (it is masked)
  const int j = t0 > last ? last & ~31 : t0;
  const int j1 = j + 16 > last ? j : j + 16;
  Ids r;
  r.id[0] = read_index(table_row, j >> c.page_log2);
  r.id[1] = c.page_log2 >= 5 ? r.id[0] : read_index(table_row, j1 >> c.page_log2);
  return r;
}

template <int D, bool GROUPS>
__device__ __forceinline__ void load_block(const Kv4Cache& c, int64_t block, int off, int t, int plus, int g, int i,
                                           Tile<D, GROUPS>& x) {
  // (block, off) and `plus` tokens, the part that is a constant of the load instructions
  const int sh = c.page_log2;
  const int64_t cb = ((block << sh) + off) * (D / 2);
  const int ng = GROUPS ? D / c.group : 1;
  const int64_t sb = ((block * ng) << sh) + off;
  const uint8_t* kp = c.codes[0] + cb + (i * (D / 2) + g * (D / 8)) + plus * (D / 2);
  const uint8_t* vp = c.codes[1] + cb + (4 * g * (D / 2) + i * (D / 32)) + plus * (D / 2);
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
    const uint8_t* vr = vp + r * (D / 2);
    if (D == 64) {
      x.v[4 * t + r][0] = *reinterpret_cast<const uint16_t*>(vr);
    } else if (D == 128) {
      x.v[4 * t + r][0] = *reinterpret_cast<const uint32_t*>(vr);
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(vr);
      x.v[4 * t + r][0] = u.x;
      x.v[4 * t + r][D / 256] = u.y;
    }
  }
  const _Float16* ks = c.scales[0] + sb;
  const _Float16* vs = c.scales[1] + sb;
  if (!GROUPS) {
    x.ks4[t] = *reinterpret_cast<const half4v*>(ks + 4 * g + plus);
    x.vs[t] = *reinterpret_cast<const half4v*>(vs + 4 * g + plus);
  } else {
#pragma unroll
    for (int n = 0; n < Tile<D, GROUPS>::NS; ++n) x.ks1[n][t] = ks[(((g * (D / 4) + 32 * n) / c.group) << sh) + i + plus];
    x.vs[t] = *reinterpret_cast<const half4v*>(vs + ((i * (D / 16) / c.group) << sh) + 4 * g + plus);
  }
}

template <int D, bool GROUPS>
__device__ __forceinline__ void load_tile(const Kv4Cache& c, Ids ids, int head, int t0, int last, int g, int i,
                                          Tile<D, GROUPS>& x) {
  const int pmask = (1 << c.page_log2) - 1;
  const int j = t0 > last ? last & ~31 : t0;
  const int id0 = (unsigned)ids.id[0] < (unsigned)c.pages ? ids.id[0] : 0;
  const int64_t block = (int64_t)id0 * c.heads + head;
  const int off = j & pmask;
  load_block<D, GROUPS>(c, block, off, 0, 0, g, i, x);
  if (c.page_log2 >= 5) {          // the tile lies in one page
    load_block<D, GROUPS>(c, block, off, 1, 16, g, i, x);
  } else {
    const int id1 = (unsigned)ids.id[1] < (unsigned)c.pages ? ids.id[1] : 0;
    load_block<D, GROUPS>(c, (int64_t)id1 * c.heads + head, 0, 1, 0, g, i, x);
  }
}

// GROUPS: several scale groups a head; PREC: what the outputs can show; ROWS
// query rows a workgroup (16 or 32), W waves (4 or 8)
template <int D, bool GROUPS, int PREC, int ROWS, int W>
__global__ __launch_bounds__(64 * W, W == 8 ? 2 : kv4_attn_waves(D, GROUPS, ROWS, PREC)) void kv4_attn_kernel(Kv4AttnArgs p) {
  constexpr int NK = D / 32;             // matrix instructions over the dims
  constexpr int NC = D / 16;             // 16-dim slices of the output
  constexpr int LD = D + 4;              // row pitch of the exchange
  constexpr int RT = ROWS / 16;
  constexpr int QT = PREC == kForBf16 ? 1 : 2;     // fp16 terms of a query, and of a scaled code
  constexpr int PT = PREC == kForF32 ? 2 : 1;      // of a probability
  // Of a probability's two terms the second is held 2^11 times as large, against values 2^-11 as large: it would
  // otherwise be 0 for probabilities under 2^-25 of the largest.  The values of 2^-11 keep their bits because they are
  // codes (one group a head: the value scales are in the probabilities) or scaled up before.
  // Value scales, where they are in the probabilities or there are two terms, are relative to a power of two, the unit,
  // that the largest so far sets.
  constexpr bool UNIT = !GROUPS || PREC == kForF32;
  constexpr int UNIT_MIN = GROUPS ? -15 : -24;     // its reciprocal an fp16 number; fp16's smallest exponent
  constexpr int UNIT_BELOW = GROUPS ? 12 : 0;      // log2 of the largest scale in units (7 times 2^12 is an fp16 number)
  typedef Tile<D, GROUPS> T;
  __shared__ float o_lds[W][16][LD];
  __shared__ float m_lds[W][16], l_lds[W][16];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, i = lane & 15;
  // heads vary fastest, then sequences, then row tiles, then parts: every
  // sequence has a first part, only long ones have late ones
  int rest = blockIdx.x / p.c.heads;
  const int head = blockIdx.x - rest * p.c.heads;
  const int b = rest % p.batch;
  rest /= p.batch;
  const int part = rest / p.tiles;
  const int row0 = (rest - part * p.tiles) * ROWS;
  const Kv4Seq q(p, b);
  if (row0 >= q.rows) return;
  // what the workgroup's first and last row see
  const int n_first = row0 / p.rep;
  const int n_last = (row0 + ROWS - 1 < q.rows ? row0 + ROWS - 1 : q.rows - 1) / p.rep;
  const int lo = q.lo(n_first), hi = q.hi(n_last);
  const int all_lo = q.lo(n_last), all_hi = q.hi(n_first);   // [all_lo, all_hi): seen by every row
  const int parts = kv4_part_count(lo, hi, p.chunk);
  if (part >= parts) return;
  const int from = kv4_part_base(lo) + part * p.chunk;
  int to = from + p.chunk;
  if (to > hi || part == p.nsplit - 1) to = hi;

  // the first tile sets out before the queries are dealt with
  const int32_t* table_row = p.table + (int64_t)b * p.width;
  constexpr int STEP = 32 * W;
  const int last = to - 1;
  int t0 = from + 32 * wave;
  const bool some = t0 < to;
  T x0, x1;
  Ids ids, ids1;
  if (some) {
    ids = load_ids(p.c, table_row, t0, last);
    ids1 = load_ids(p.c, table_row, t0 + STEP, last);
    load_tile<D, GROUPS>(p.c, ids, head, t0, last, g, i, x0);
  }

  // queries, 16 lanes a row as in the output: rotate, scale to [1, 2) by a power of two (kept in qf), round, and
  // through LDS into the right operand's layout
  constexpr int QP = D + 8;              // row pitch, 16-bit elements
  static_assert(RT * QT * QP * 2 <= W * LD * 4, "the queries fit the exchange");
  uint16_t* q_lds = reinterpret_cast<uint16_t*>(o_lds);
  float qf[RT];
  int my_lo[RT];
  unsigned my_span[RT];        // the row's tokens: [my_lo, my_lo + my_span)
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int mine = row0 + 16 * rt + i;
    const int n_mine = (mine < q.rows ? mine : q.rows - 1) / p.rep;
    my_lo[rt] = q.lo(n_mine);
    const int my_end = q.hi(n_mine) < to ? q.hi(n_mine) : to;
    my_span[rt] = my_end > my_lo[rt] ? my_end - my_lo[rt] : 0;
    if (W > 4 && wave >= 4) continue;      // four waves are 16 rows
    const int qrow = threadIdx.x >> 4;
    const int la = p.c.rotate ? kv4_logical<16>(lane) : lane & 15;
    const int row = row0 + 16 * rt + qrow;
    const int n = row < q.rows ? row / p.rep : 0;
    float w[NC];
    if (row < q.rows) {
      load_vec_any<NC>(p.dtype, p.q, (int64_t)(q.s0 + n) * p.q_stride + (head * p.rep + row - n * p.rep) * D + la * NC, w);
    } else {
#pragma unroll
      for (int e = 0; e < NC; ++e) w[e] = 0.0f;
    }
    if (p.c.rotate) {
      uint32_t sg[NC];
      load_signs<NC>(p.c.signs, la * NC, sg);
#pragma unroll
      for (int e = 0; e < NC; ++e) w[e] = flip(w[e], sg[e]);
      fwht_lanes<NC, 16>(w, la);
      const float nf = kv4_norm<D>() * kv4_tau(la);
#pragma unroll
      for (int e = 0; e < NC; ++e) w[e] *= nf;
    }
    float mx = 0.0f;
#pragma unroll
    for (int e = 0; e < NC; ++e) mx = fmaxf(mx, fabsf(w[e]));
    uint32_t u = umax_dpp<kQuadXor1>(__float_as_uint(mx));
    u = umax_dpp<kQuadXor2>(u);
    u = umax_dpp<kRowHalfMirror>(u);
    const int ex = row_exponent(__uint_as_float(umax_dpp<kRowMirror>(u)));
    // never 0, which would make NaN of a masked score; products of [1, 2) with keys are far below 2^100, so a factor
    // this small makes all of them 0
    if ((lane & 15) == 0) l_lds[rt][qrow] = fmaxf(ldexpf(p.scale, ex) * kLog2e, 0x1p-126f);
    // dim d of a row at place 8 (d / 8) + (the e with kOrder[e] = d % 8)
    constexpr int EN = NC < 8 ? NC : 8;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      uint16_t* to_row = q_lds + ((rt * QT + t) * 16 + qrow) * QP;
#pragma unroll
      for (int c = 0; c < (NC + 7) / 8; ++c) {
        uint16_t h[EN];
#pragma unroll
        for (int e = 0; e < EN; ++e) {
          float& y = w[8 * c + e];
          if (t == 0) y = ldexpf(y, -ex);
          const _Float16 r = (_Float16)y;
          y -= (float)r;
          h[e] = __builtin_bit_cast(uint16_t, r);
        }
        if (NC >= 8) {
          u32x4 v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = (uint32_t)h[kOrder[2 * e] % EN] | ((uint32_t)h[kOrder[2 * e + 1] % EN] << 16);
          *reinterpret_cast<u32x4*>(to_row + la * NC + 8 * c) = v;
        } else {
          // dims 4 la .. 4 la + 3: the even or the odd places of their eight
#pragma unroll
          for (int e = 0; e < 4; ++e) to_row[8 * (la >> 1) + 2 * e + (la & 1)] = h[e % EN];
        }
      }
    }
  }
  __syncthreads();
  half8v qh[RT][QT][NK];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    qf[rt] = l_lds[rt][i];
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
      for (int c = 0; c < NK; ++c)
        qh[rt][t][c] = *reinterpret_cast<const half8v*>(q_lds + ((rt * QT + t) * 16 + i) * QP + g * (D / 4) + 8 * c);
  }

  f32x4 acc[RT][NC], accl[RT];
  float m[RT];
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[rt][c] = zero;
    accl[rt] = zero;
    m[rt] = -__builtin_inff();
  }
  int vexp = UNIT_MIN;                   // acc is in units of 2^vexp
  float vcap = 0.0f, vinv = 1.0f;        // the largest scale that the unit is for; 2^-vexp
  const half4v zero4 = {(_Float16)0, (_Float16)0, (_Float16)0, (_Float16)0};
  const half2v down = {(_Float16)0x1p-11f, (_Float16)0x1p-11f};
  const half8v ones_h = {(_Float16)1, (_Float16)1, (_Float16)1, (_Float16)1, (_Float16)1, (_Float16)1, (_Float16)1, (_Float16)1};

  auto step = [&](const T& x, int t0) {
    // S^T
    f32x4 s[RT][2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) s[rt][t] = zero;
#pragma unroll
      for (int c = 0; c < NK; ++c) {
        half2v h[4], h1[4];
        codes8(x.k[t][c], h);
        if (GROUPS) {
          const _Float16 sc = (c < 4 ? x.ks1[0] : x.ks1[T::NS - 1])[t];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const half2v y = h[u] * (half2v){sc, sc};
            if (QT == 2) h1[u] = __builtin_elementwise_fma(h[u], (half2v){sc, sc}, -y);   // what the rounding left
            h[u] = y;
          }
        }
        const half8v k = join8(h);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          if (GROUPS && QT == 2) s[rt][t] = mma(join8(h1), qh[rt][0][c], s[rt][t]);
          if (QT == 2) s[rt][t] = mma(k, qh[rt][QT - 1][c], s[rt][t]);
          s[rt][t] = mma(k, qh[rt][0][c], s[rt][t]);
        }
      }
    }
    // a poisoned token has NaN scales: its score carries that to the rows that see it, its value must not
    half4v vs[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) vs[t] = __builtin_elementwise_max(x.vs[t], zero4);
    const bool edge = t0 < all_lo || t0 + 32 > (all_hi < to ? all_hi : to);
    if (edge) {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int j = t0 + 16 * (u >> 2) + 4 * g + (u & 3);
        if (j < lo || j >= to) vs[u >> 2][u & 3] = (_Float16)0;    // never written: may hold anything
      }
    }
    half4v vd[2] = {zero4, zero4};      // 2^-11 of the scales
    if (UNIT) {
      const half4v v4 = __builtin_elementwise_max(vs[0], vs[1]);
      const half2v v2 = __builtin_elementwise_max((half2v){v4[0], v4[1]}, (half2v){v4[2], v4[3]});
      const float vm = fmaxf((float)v2[0], (float)v2[1]);
      if (__builtin_amdgcn_ballot_w64(vm > vcap)) {
        uint32_t u = __float_as_uint(max_over_g(vm));
        if (GROUPS) {        // lanes of a row hold different groups
          u = umax_dpp<kQuadXor1>(u);
          u = umax_dpp<kQuadXor2>(u);
          u = umax_dpp<kRowHalfMirror>(u);
          u = umax_dpp<kRowMirror>(u);
        }
        int e = __builtin_amdgcn_readfirstlane(__builtin_amdgcn_frexp_expf(__uint_as_float(u))) - UNIT_BELOW;
        if (e < UNIT_MIN) e = UNIT_MIN;
        if (e > vexp) {
          const float f = ldexpf(1.0f, vexp - e);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int c = 0; c < NC; ++c) acc[rt][c] *= f;
          vexp = e;
        }
        vcap = ldexpf(1.0f, vexp + UNIT_BELOW);
        vinv = ldexpf(1.0f, -vexp);
      }
      if (GROUPS) {
        const _Float16 up = (_Float16)vinv;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          vs[t] = vs[t] * (half4v){up, up, up, up};
          vd[t] = vs[t] * (half4v){down[0], down[0], down[0], down[0]};
        }
      }
    }
    // probabilities
    half8v pv[RT][PT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float z[8];      // scores of row i at tokens t0 + 16 t + 4 g + r
#pragma unroll
      for (int u = 0; u < 8; ++u)
        z[u] = !GROUPS ? s[rt][u >> 2][u & 3] * (float)x.ks4[u >> 2][u & 3] : s[rt][u >> 2][u & 3];
      if (edge) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int j = t0 + 16 * (u >> 2) + 4 * g + (u & 3);
          z[u] = (unsigned)(j - my_lo[rt]) < my_span[rt] ? z[u] : -__builtin_inff();
        }
      }
      float mx = z[0];
#pragma unroll
      for (int u = 1; u < 8; ++u) mx = fmaxf(mx, z[u]);
      mx *= qf[rt];
      if (__builtin_amdgcn_ballot_w64(mx > m[rt] + kMaxSlack)) {
        const float mn = fmaxf(m[rt], max_over_g(mx));
        const float f = mn > m[rt] ? exp2f(m[rt] - mn) : 1.0f;
        m[rt] = mn;
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[rt][c] *= f;
        accl[rt] *= f;
      }
      const float mu = (m[rt] == -__builtin_inff() ? 0.0f : m[rt]) - kLift;
      float pr[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) pr[u] = __builtin_amdgcn_exp2f(fmaf(z[u], qf[rt], -mu));
      // the softmax sum takes them as rounded
      half8v ph[PT];
#pragma unroll
      for (int t = 0; t < PT; ++t) {
#pragma unroll
        for (int u = 0; u < 8; ++u) ph[t][u] = (_Float16)(t ? (pr[u] - (float)ph[0][u]) * 0x1p11f : pr[u]);
        accl[rt] = mma(t ? ones_h * (_Float16)0x1p-11f : ones_h, ph[t], accl[rt]);
        pv[rt][t] = ph[t];
      }
      if (!GROUPS) {
        // multiplied in fp32: a scale far larger than the others, which some row may not even see, would make fp16's
        // subnormals or zeros of them
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          float y = pr[u] * ((float)vs[u >> 2][u & 3] * vinv);
          if (PT == 2) asm("" : "+v"(y));      // one fp32 number for both terms: a mixed-precision fma rounds its own way
          pv[rt][0][u] = (_Float16)y;
          if (PT == 2) pv[rt][PT - 1][u] = (_Float16)((y - (float)pv[rt][0][u]) * 0x1p11f);
        }
      }
    }
    // O^T
#pragma unroll
    for (int bb = 0; bb < NC / 2; ++bb) {
      half2v vv[2][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        codes_of_two(x.v[2 * j][bb >> 2], x.v[2 * j + 1][bb >> 2], bb & 3, vv[0][j], vv[1][j]);
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const int c = 2 * bb + d;
        half2v v1[4], v2[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const half2v sc = {vs[j >> 1][2 * (j & 1)], vs[j >> 1][2 * (j & 1) + 1]};
          const half2v sd = {vd[j >> 1][2 * (j & 1)], vd[j >> 1][2 * (j & 1) + 1]};
          if (PT == 2) v2[j] = vv[d][j] * (GROUPS ? sd : down);
          if (GROUPS) {
            const half2v y = vv[d][j] * sc;
            if (QT == 2) v1[j] = __builtin_elementwise_fma(vv[d][j], sc, -y);
            vv[d][j] = y;
          }
        }
        const half8v v = join8(vv[d]);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          if (GROUPS && QT == 2) acc[rt][c] = mma(join8(v1), pv[rt][0], acc[rt][c]);
          if (PT == 2) acc[rt][c] = mma(join8(v2), pv[rt][PT - 1], acc[rt][c]);
          acc[rt][c] = mma(v, pv[rt][0], acc[rt][c]);
        }
      }
    }
  };

  // two tiles in registers: one at work, the next on its way; the page ids of a third
  if (some) {
    for (;;) {
      ids = load_ids(p.c, table_row, t0 + 2 * STEP, last);
      load_tile<D, GROUPS>(p.c, ids1, head, t0 + STEP, last, g, i, x1);
      step(x0, t0);
      t0 += STEP;
      if (t0 >= to) break;
      ids1 = load_ids(p.c, table_row, t0 + 2 * STEP, last);
      load_tile<D, GROUPS>(p.c, ids, head, t0 + STEP, last, g, i, x0);
      step(x1, t0);
      t0 += STEP;
      if (t0 >= to) break;
    }
  }

  // join the waves, 16 rows at a time: lane (g, i) holds dims [g D/4, (g+1) D/4) of row i
  __syncthreads();           // the exchange held the queries
  const float unit = UNIT ? ldexpf(1.0f, vexp) : 1.0f;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    if (rt) __syncthreads();
    if (g == 0) m_lds[wave][i] = m[rt];
    __syncthreads();
    float top = m_lds[0][i];
#pragma unroll
    for (int w = 1; w < W; ++w) top = fmaxf(top, m_lds[w][i]);
    const float f = m[rt] == -__builtin_inff() ? 0.0f : exp2f(m[rt] - top);
    const float fu = f * unit;
    if (g == 0) l_lds[wave][i] = accl[rt][0] * f;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int c = 0; c < NC; c += 4)
        *reinterpret_cast<f32x4*>(&o_lds[wave][i][(4 * g + r) * NC + c]) =
            (f32x4){acc[rt][c][r] * fu, acc[rt][c + 1][r] * fu, acc[rt][c + 2][r] * fu, acc[rt][c + 3][r] * fu};
    __syncthreads();
    if (W > 4 && wave >= 4) continue;
    // 16 lanes a row, D/16 consecutive dims each
    const int orow = threadIdx.x >> 4;
    const int la = kv4_logical<16>(lane);
    float y[NC], l = 0.0f, mt = m_lds[0][orow];
#pragma unroll
    for (int e = 0; e < NC; ++e) y[e] = 0.0f;
#pragma unroll
    for (int v = 0; v < W; ++v) {
      l += l_lds[v][orow];
      mt = fmaxf(mt, m_lds[v][orow]);
#pragma unroll
      for (int e = 0; e < NC; e += 4) {
        const f32x4 r = *reinterpret_cast<const f32x4*>(&o_lds[v][orow][la * NC + e]);
#pragma unroll
        for (int u = 0; u < 4; ++u) y[e + u] += r[u];
      }
    }
    const int r2 = row0 + 16 * rt + orow;
    const bool store = r2 < q.rows;
    const int n2 = store ? r2 / p.rep : 0;
    const int64_t out_row = (int64_t)(q.s0 + n2) * p.q_heads + head * p.rep + (store ? r2 - n2 * p.rep : 0);
    if (parts > 1 && p.nsplit > 1) {
      if (store) {
        const int64_t at = out_row * p.nsplit + part;
        store_vec<kDtF32, NC>(p.part_o + at * D + la * NC, y);
        if (la == 0) p.part_ml[at] = make_float2(mt, l);
      }
    } else {
      finish_row<D>(p.c.rotate, p.c.signs, l, la, y);
      if (store) store_vec_any<NC>(p.dtype, p.out, out_row * D + la * NC, y);
    }
  }
}

// Joins the parts of output rows.  GROUPS 16-lane groups of a workgroup share
// a row and take its parts in turn; LDS adds the groups up, the first of them
// rotates back.  One group a row where parts are few (a wave's work is then all
// loads, and a workgroup does 16 rows), all 16 where they are many.
template <int D, int GROUPS>
__global__ __launch_bounds__(256) void kv4_join_kernel(Kv4AttnArgs p) {
  constexpr int NC = D / 16;
  __shared__ float o_lds[GROUPS][D + 4];
  __shared__ float l_lds[GROUPS], m_lds[GROUPS];
  const int lane = threadIdx.x & 63;
  const int grp = (threadIdx.x >> 4) % GROUPS;
  const int la = kv4_logical<16>(lane);
  const int b = blockIdx.y;
  const int at_row = blockIdx.x * (16 / GROUPS) + (threadIdx.x >> 4) / GROUPS;
  const int n = at_row / p.q_heads, q_head = at_row - n * p.q_heads;
  const Kv4Seq q(p, b);
  const bool valid = n < q.news && n < p.max_new;
  const int64_t out_row = (int64_t)(q.s0 + (valid ? n : 0)) * p.q_heads + q_head;
  // its row tile's parts (with one, the row is finished)
  int parts = 1;
  if (valid) {
    const int row0 = (n * p.rep + q_head % p.rep) / p.rows * p.rows;
    const int row1 = row0 + p.rows < q.rows ? row0 + p.rows : q.rows;
    parts = kv4_part_count(q.lo(row0 / p.rep), q.hi((row1 - 1) / p.rep), p.chunk);
    if (parts > p.nsplit) parts = p.nsplit;
  }
  if (GROUPS > 1 && parts == 1) return;      // the whole workgroup
  const int64_t first = out_row * p.nsplit;
  // four parts asked for at once, against a maximum of the group's own
  float w[NC], l = 0.0f, m = -__builtin_inff();
#pragma unroll
  for (int e = 0; e < NC; ++e) w[e] = 0.0f;
  if (parts > 1) {
    for (int s0 = grp; s0 < parts; s0 += 4 * GROUPS) {
      float2 v[4];
      float o[4][NC];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t at = first + (s0 + u * GROUPS < parts ? s0 + u * GROUPS : s0);
        v[u] = p.part_ml[at];
        load_vec<kDtF32, NC>(p.part_o + at * D + la * NC, o[u]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (s0 + u * GROUPS >= parts) continue;
        const float mn = fmaxf(m, v[u].x);
        const float f0 = m == -__builtin_inff() ? 0.0f : exp2f(m - mn);
        const float f1 = v[u].x == -__builtin_inff() ? 0.0f : exp2f(v[u].x - mn);
        m = mn;
        l = l * f0 + v[u].y * f1;
#pragma unroll
        for (int e = 0; e < NC; ++e) w[e] = fmaf(o[u][e], f1, w[e] * f0);
      }
    }
  }
  if (GROUPS > 1) {
    store_vec<kDtF32, NC>(&o_lds[grp][la * NC], w);
    if (la == 0) {
      l_lds[grp] = l;
      m_lds[grp] = m;
    }
    __syncthreads();
    if (grp >= 4) return;      // the first wave goes on (all of it: the exchanges need whole rows)
    float top = m_lds[0];
#pragma unroll
    for (int s = 1; s < GROUPS; ++s) top = fmaxf(top, m_lds[s]);
#pragma unroll
    for (int e = 0; e < NC; ++e) w[e] = 0.0f;
    l = 0.0f;
#pragma unroll 4
    for (int s = 0; s < GROUPS; ++s) {
      const float f = m_lds[s] == -__builtin_inff() ? 0.0f : exp2f(m_lds[s] - top);
      l = fmaf(l_lds[s], f, l);
#pragma unroll
      for (int e = 0; e < NC; ++e) w[e] = fmaf(o_lds[s][la * NC + e], f, w[e]);
    }
  }
  finish_row<D>(p.c.rotate, p.c.signs, l, la, w);
  if (grp == 0 && parts > 1) store_vec_any<NC>(p.dtype, p.out, out_row * D + la * NC, w);
}

// Which kernel, and into how many parts of the token axis.
//
// Rows: 16 a workgroup of the kernel above, and fp16 calls of more than 16 rows a
// key/value head 32 where that still makes two workgroups a CU (the codes of a
// tile are then made fp16 once for both halves: 1024 tokens, 32 heads on 8, over
// 4096 197 against 224 us; where there are fewer, twice the workgroups wait less:
// 64 sequences of 3 new tokens, 64 heads on 8, 48 against 60).  Up to 16 rows half
// of such a workgroup would be empty (64 sequences of up to 8192 tokens, one new
// token, 32 on 8: 81 against 110).
//
// bf16 calls of more than 64 rows a key/value head and enough work take the
// prompt kernel, whose fewer, larger workgroups cost less a score but start
// later: enough is 16-row tiles times tokens past 8192 dim (32 heads on 8 of 128
// dims, prompt kernel against 16 rows: 4 sequences, 64 new tokens over 4000 43
// against 50 us; 1 of 256 over 2048 43 against 26, 1 of 512 alone 30 against 16, 1
// of 64 over 8192 45 against 32; 64 dims, 4 of 32 over 4000 22 against 26, 1 of 32
// over 8192 22 against 18; up to 64 rows, 64 sequences of 10 new tokens 150 against
// 74).  128 rows of it, or 256 for 128 dims and more than 128 rows (2048 tokens
// over 8192: 276 against 292 us; 64 dims lose the third workgroup a CU, 127 against
// 101 us, and 256 dims the registers).  Its keys and values are rounded to fp16,
// which an fp16 output would show (its error 5.5e-4 where the rounding of the
// output alone is 2.1e-4, against 2.4e-4 here, at 372 us where this takes 407).
//
// Parts: two workgroups a CU for one sequence, whose parts are all alike (131071
// tokens, 8 heads: 35.7 us; three a CU 37.6, four 39.9, one and a half 40.8),
// two and a half for several, whose lengths differ (64 sequences of 1100 to 8192
// tokens: 77.9 us; two a CU 84.6, five 80.5); no part under 256 tokens (two tiles
// a wave), or 512 of the prompt kernel, which gets as many workgroups as run at
// once.  Several row tiles of several sequences share their tokens in L2 and are
// bound by waiting: five workgroups a CU and no part under 512, where three run at
// once (12 sequences of up to 6000 tokens, 5 new ones each, 40 heads on 8, two
// groups a head: 29.0 us; four a CU 30.6, two and a half 36.9, six 32.1; but 38.5
// against 32.5 for 256 dims, of which two run).  Sequences of up to 1024 tokens,
// no more than one workgroup a CU, are not divided: 8 waves take one (4 tiles a
// wave) and no second launch follows (1024 tokens of one sequence: 10.5 against
// 12.7 us; up to 2048 of 16, 64 dims: 14.3 undivided, 13.4 in parts).
void kv4_attention_plan(Kv4AttnArgs* a) {
  const int64_t rows = (int64_t)a->max_new * a->rep;
  int64_t span = a->max_len;
  if (a->window > 0 && (int64_t)a->window + a->max_new + 31 < span) span = (int64_t)a->window + a->max_new + 31;
  const int64_t pairs = (int64_t)a->batch * a->c.heads;
  a->rows = 16;
  if (a->dtype == kDtBf16 && rows > 64 && pairs * ((rows + 15) / 16) > 8192 * (int64_t)a->c.dim / (span > 0 ? span : 1))
    a->rows = a->c.dim == 128 && rows > 128 ? 256 : 128;
  if (a->dtype == kDtF16 && rows > 16 && a->c.dim <= 128 && pairs * ((rows + 31) / 32) >= 512) a->rows = 32;
  a->tiles = (int)((rows + a->rows - 1) / a->rows);
  const int64_t segments = pairs * a->tiles;
  const int prec = a->dtype == kDtBf16 ? kForBf16 : a->dtype == kDtF16 ? kForF16 : kForF32;
  const bool several = a->rows == 16 && a->tiles > 1 && kv4_attn_waves(a->c.dim, a->c.group != a->c.dim, 16, prec) == 3;
  const int64_t least = a->rows >= 128 || several ? 512 : 256;
  int64_t want = a->rows == 256 ? 256 : a->rows == 128 || a->batch == 1 ? 512 : several ? 1280 : 640;
  a->waves = 4;
  if (a->rows == 16 && segments <= 256 && span <= 1024) {
    a->waves = 8;
    want = 1;
  }
  int64_t n = segments > 0 ? (want + segments - 1) / segments : 1;
  const int64_t most = (span + least - 1) / least;
  if (n > most) n = most;
  if (n < 1) n = 1;
  int64_t chunk = ((span + n - 1) / n + 127) / 128 * 128;
  if (chunk < least) chunk = least;
  n = (span + chunk - 1) / chunk;
  a->nsplit = (int)(n < 1 ? 1 : n);
  a->chunk = a->nsplit == 1 ? kKv4MaxLen : (int)chunk;
  a->groups = segments * a->nsplit;
}

template <int D, bool GROUPS, int PREC>
static void attn2(const Kv4AttnArgs& a, hipStream_t s) {
  constexpr int MORE = D <= 128 && PREC == kForF16 ? 32 : 16;
  const dim3 g((unsigned)a.groups);
  if (a.waves == 8) hipLaunchKernelGGL((kv4_attn_kernel<D, GROUPS, PREC, 16, 8>), g, dim3(512), 0, s, a);
  else if (a.rows == MORE) hipLaunchKernelGGL((kv4_attn_kernel<D, GROUPS, PREC, MORE, 4>), g, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((kv4_attn_kernel<D, GROUPS, PREC, 16, 4>), g, dim3(256), 0, s, a);
}

template <int D, bool GROUPS>
static void attn3(const Kv4AttnArgs& a, hipStream_t s) {
  if (a.dtype == kDtF32) attn2<D, GROUPS, kForF32>(a, s);
  else if (a.dtype == kDtF16) attn2<D, GROUPS, kForF16>(a, s);
  else attn2<D, GROUPS, kForBf16>(a, s);
}

template <int D>
static void attn1(const Kv4AttnArgs& a, hipStream_t s) {
  if (a.rows >= 128) launch_kv4_prompt(a, s);
  else if (a.c.group == D) attn3<D, false>(a, s);
  else attn3<D, true>(a, s);
  if (a.nsplit > kFewParts)
    hipLaunchKernelGGL((kv4_join_kernel<D, 16>), dim3((unsigned)(a.max_new * a.q_heads), a.batch), dim3(256), 0, s, a);
  else if (a.nsplit > 1)
    hipLaunchKernelGGL((kv4_join_kernel<D, 1>), dim3((unsigned)((a.max_new * a.q_heads + 15) / 16), a.batch),
                       dim3(256), 0, s, a);
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
