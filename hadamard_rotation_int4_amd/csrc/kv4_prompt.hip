// Attention over the 4-bit key/value cache for many query rows (prompts and
// chunks of prompts), bf16 queries.  The mathematics is kv4_attention.hip's;
// here it is the matrix products that count, so a workgroup shares each tile's
// codes-to-fp16 work among 128 or 256 query rows through LDS.
//
// One workgroup of 4 or 8 waves takes 32 query rows a wave of one (sequence,
// key/value head), row = new token * rep + head of the group, and walks over
// 64-token tiles.  Each wave computes, on 32x32x16 instructions,
//   S^T = K q'^T (rows: tokens),   O^T = V^T P^T (rows: dims):
// S^T leaves query row n = lane % 32 in the lane, with tokens
// 8 (r / 4) + 4 h + r % 4 in register r (h = lane / 32), which is what the
// second product wants as its right operand when its contraction slots
// (h, i) stand for tokens 8 (i / 4) + 4 h + i % 4.  So probabilities never
// leave their lane, and the softmax needs one exchange (between the two halves
// of a wave), and that only when the running maximum moves.
//
// Queries are scaled by the softmax scale and log2(e) before they are rounded, so
// that scores come out as exponents.  Keys, scaled, and queries are rounded to
// fp16: a score is good to 2^-11 of its terms' sizes (of keys that are all alike
// the rounding does not average out), where the row kernel holds keys of one
// group exactly.  Probabilities are fp16 too, 2^-12 of those down to 2^-25 of the
// largest (kLift).
//
// LDS holds scaled fp16, in 16-byte pieces that a wave reads contiguously:
//   keys    [dim / 8][64 tokens] pieces of 8 dims (in nibble order; the
//           queries are laid out to match), one piece of padding a row so that
//           the four rows a wave writes at once fall into different banks;
//   values  [8 octets][dim] pieces of 8 tokens, octet 2 t + h holding the
//           tokens of slots (h, .) of 16-token step t; a piece's place among
//           the dims is the transposed (dim % (dim/16), dim / (dim/16)), so
//           that 16 lanes that hold neighbouring dims write contiguously.
// Two buffers of each.  A turn of the loop makes the scores of tile t + 1 while
// the softmax works on those of tile t, then adds tile t's values while the keys
// of t + 2 and the values of t + 1 become fp16; one barrier a turn.  With 8
// waves four deal with the keys and four with the values.
//
// 2048 tokens, 32 heads on 8, 128 dims, over 8192, 8 waves: 272 us, 0.88 PFLOP/s
// where a large library product reaches 1.23; the matrix pipe is busy 37% of the
// time, vector instructions 46%.  There is one workgroup a CU, and the first rows' see
// 6208 tokens where the last rows' see 8192, so the mean is 0.88 of the longest.
// Inside one (4 waves, 290 us): without the fp16 work, the exponentials and the LDS
// reads the loop takes 199, the library product's rate; making fp16 costs 65 (8 waves
// halve that), the LDS reads 22, the exponentials 16.
// At 64 dims a score costs half the products and the same softmax: 210 vector
// instructions a tile and wave (32 exponentials of 16 cycles among them) beside 16
// matrix ones of 32.  6 ragged sequences of up to 1500 tokens, a window of 1024: 94 us
// a call, vector instructions 58% of the time and two waves a SIMD where three fit:
// with at most 17 tiles, what comes before and after the loop counts.  Outputs
// used to go through LDS, 16 rows at a time; turned back in registers like the
// queries they cost 700 fewer instructions a wave, 94.4 against 98.4 us a call.
//
// Heads vary fastest over the grid, so that with 8 heads the workgroups of one
// head share an XCD's L2; the last rows, which see most, go first.
#include "kv4_attention.h"

namespace hr {

constexpr int kPromptTokens = 64;           // of a tile

typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16 mma32(half8v a, half8v b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// One thread's share of a tile on its way to LDS: a quarter of one token's key,
// and dim / 16 dims of four tokens' values, with their scales.  Wave w's shares
// are of the tile's 16-token block w: one page.
template <int D>
struct KeyShare {
  static constexpr int NS = D == 256 ? 2 : 1;           // 32-dim spans with scales of their own
  uint32_t k[D / 32];
  _Float16 s[NS];
};
template <int D>
struct ValueShare {
  static constexpr int NV = (D + 127) / 128;            // dwords a token
  uint32_t v[4][NV];
  half4v s;
};

// Where the codes (bytes) and scales (elements) of the 16 tokens from token j, a
// multiple of 16, start in either of the cache's arrays; past the last token,
// any block of the sequence (it is masked).
struct Place {
  int64_t codes, scales;
};
template <int D>
__device__ __forceinline__ Place place_of(const Kv4Cache& c, const int32_t* table_row, int head, int j, int last) {
  if (j > last) j = last & ~15;
  int id = read_index(table_row, j >> c.page_log2);
  if ((unsigned)id >= (unsigned)c.pages) id = 0;
  const int off = j & ((1 << c.page_log2) - 1);
  const int64_t block = (int64_t)id * c.heads + head;
  return {((block << c.page_log2) + off) * (D / 2), ((block * (D / c.group)) << c.page_log2) + off};
}

template <int D>
__device__ __forceinline__ void load_keys(const Kv4Cache& c, Place at, int lane, KeyShare<D>& x) {
  const int kt = lane >> 2, kp = lane & 3;              // token of the block, quarter
  const uint8_t* kk = c.codes[0] + at.codes + (kt * (D / 2) + kp * (D / 8));
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
  const _Float16* sc = c.scales[0] + at.scales;
#pragma unroll
  for (int n = 0; n < KeyShare<D>::NS; ++n) x.s[n] = sc[(((kp * (D / 4) + 32 * n) / c.group) << c.page_log2) + kt];
}

template <int D>
__device__ __forceinline__ void load_values(const Kv4Cache& c, Place at, int lane, ValueShare<D>& x) {
  const int vq = lane >> 4, va = lane & 15;             // token quad of the block, dims
  const uint8_t* vc = c.codes[1] + at.codes + (4 * vq * (D / 2) + va * (D / 32));
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint8_t* vv = vc + r * (D / 2);
    if (D == 64) {
      x.v[r][0] = *reinterpret_cast<const uint16_t*>(vv);
    } else if (D == 128) {
      x.v[r][0] = *reinterpret_cast<const uint32_t*>(vv);
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(vv);
      x.v[r][0] = u.x;
      x.v[r][ValueShare<D>::NV - 1] = u.y;
    }
  }
  x.s = *reinterpret_cast<const half4v*>(c.scales[1] + at.scales + ((va * (D / 16) / c.group) << c.page_log2) + 4 * vq);
}

template <int D>
struct PromptLds {
  static constexpr int KROW = kPromptTokens * 16 + 16;  // bytes of a row of key pieces
  static constexpr int KEYS = D / 8 * KROW;
  static constexpr int VALUES = kPromptTokens / 8 * D * 16;
  static constexpr int ALL = 2 * KEYS + 2 * VALUES;     // two key buffers, two value buffers
};

// The shares to fp16 and into a buffer.
template <int D>
__device__ __forceinline__ void store_keys(const KeyShare<D>& x, char* buf, int wave, int lane) {
  const int kt = lane >> 2, kp = lane & 3;
#pragma unroll
  for (int n = 0; n < D / 32; ++n) {
    half2v h[4];
    codes8(x.k[n], h);
    const _Float16 s = x.s[KeyShare<D>::NS == 1 ? 0 : n / 4];
#pragma unroll
    for (int u = 0; u < 4; ++u) h[u] = h[u] * (half2v){s, s};
    *reinterpret_cast<half8v*>(buf + (kp * (D / 32) + n) * PromptLds<D>::KROW + (16 * wave + kt) * 16) = join8(h);
  }
}

// [lo, to): tokens that some row of the tile sees; values of others may be
// anything and become 0.
template <int D>
__device__ __forceinline__ void store_values(const ValueShare<D>& x, char* buf, int wave, int lane, int j0, int lo, int to) {
  const int vq = lane >> 4, va = lane & 15;
  const half4v zero4 = {(_Float16)0, (_Float16)0, (_Float16)0, (_Float16)0};
  half4v vs = __builtin_elementwise_max(x.s, zero4);    // a poisoned token's NaN is in its score
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int j = j0 + 4 * vq + r;
    vs[r] = j < lo || j >= to ? (_Float16)0 : vs[r];
  }
  const half2v s01 = {vs[0], vs[1]}, s23 = {vs[2], vs[3]};
  char* vb = buf + (2 * wave + (vq & 1)) * (D * 16) + (vq >> 1) * 8;
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

// w := H_{2 E} w over a lane's E values and those of the lane 32 on.
template <int E>
__device__ __forceinline__ void fwht_halves(float* w, int h) {
  fwht_regs<E>(w);
  const float bh = h ? -1.0f : 1.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(w[e]), __float_as_uint(w[e]), false, false);
    w[e] = fmaf(__uint_as_float(s[1]), bh, __uint_as_float(s[0]));
  }
}

// Bits [0, n) set, n clamped to 0..32.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

template <int D, int W>
__global__ __launch_bounds__(64 * W, D == 256 ? 1 : 2) void kv4_prompt_kernel(Kv4AttnArgs p) {
  typedef PromptLds<D> L;
  constexpr int NC = D / 16, NB = D / 32;
  // The products start from minus the running maximum instead of 0 and need no subtraction (128 dims, the case
  // above: 278 against 285 us).  At 64 dims the sixteen registers that holds cost the third workgroup a CU or spills
  // (97.0 against 94.7 us, the ragged case), and scores are made relative after the products.
  constexpr bool RELATIVE = D != 64;
  __shared__ __attribute__((aligned(16))) char lds[L::ALL];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5, n = lane & 31;
  const int head = blockIdx.x % p.c.heads;
  int rest = blockIdx.x / p.c.heads;
  const int part = rest % p.nsplit;
  rest /= p.nsplit;
  const int b = rest / p.tiles;
  const int tile = p.tiles - 1 - (rest - b * p.tiles);
  const Kv4Seq q(p, b);
  constexpr int ROWS = 32 * W;
  const int row0 = tile * ROWS;
  if (row0 >= q.rows) return;
  // what the workgroup's rows see
  const int row_end = row0 + ROWS < q.rows ? row0 + ROWS : q.rows;
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
  const int all_lo = q.lo(w_last), all_hi = q.hi(w_first);
  const int row = wrow0 + n;
  const bool valid = row < q.rows;
  const int n_mine = valid ? row / p.rep : w_last;
  const int q_head = head * p.rep + (valid ? row - n_mine * p.rep : 0);     // a row past the last reads one that is there
  const int my_lo = q.lo(n_mine), my_end = valid ? (q.hi(n_mine) < to ? q.hi(n_mine) : to) : 0;

  const int32_t* table_row = p.table + (int64_t)b * p.width;
  char* const kbuf = lds;
  char* const vbuf = lds + 2 * L::KEYS;
  const int last = to - 1, blk = 16 * (wave & 3);
  // of 8 waves four deal with the keys and four with the values
  const bool does_k = W == 4 || wave < 4, does_v = W == 4 || wave >= 4;
  // the first tiles set out before the queries are dealt with
  KeyShare<D> xk0, xk1, xk;
  ValueShare<D> xv0, xv;
  Place ahead = {0, 0};          // of the tile whose keys were asked for last
  if (from < to) {
    const Place p0 = place_of<D>(p.c, table_row, head, from + blk, last);
    const Place p1 = place_of<D>(p.c, table_row, head, from + kPromptTokens + blk, last);
    ahead = place_of<D>(p.c, table_row, head, from + 2 * kPromptTokens + blk, last);
    if (does_k) {
      load_keys<D>(p.c, p0, lane, xk0);
      load_keys<D>(p.c, p1, lane, xk1);
      load_keys<D>(p.c, ahead, lane, xk);
    }
    if (does_v) {
      load_values<D>(p.c, p0, lane, xv0);
      load_values<D>(p.c, p1, lane, xv);
    }
  }

  // queries: lane (h, n) holds dims 16 c + 8 h + e of row n
  half8v qf[NC];
  float qs;
  {
    constexpr int E = D / 2;
    float w[E];
    const int64_t at = (int64_t)(q.s0 + n_mine) * p.q_stride + q_head * D;
#pragma unroll
    for (int c = 0; c < NC; ++c) load_vec<kDtBf16, 8>(reinterpret_cast<const uint16_t*>(p.q) + at + 16 * c + 8 * h, w + 8 * c);
    float norm = p.scale;
    if (norm > 0x1p60f) {        // goes with tiny queries: half of it to them, so that no factor overflows
#pragma unroll
      for (int e = 0; e < E; ++e) w[e] *= 0x1p64f;
      norm *= 0x1p-64f;
    }
    norm *= kLog2e;
    if (p.c.rotate) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        uint32_t sg[8];
        load_signs<8>(p.c.signs, 16 * c + 8 * h, sg);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[8 * c + e] = flip(w[8 * c + e], sg[e]);
      }
      fwht_halves<E>(w, h);
      norm *= kv4_norm<D>();
    }
    float mx = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) mx = fmaxf(mx, fabsf(w[e]));
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(mx), __float_as_uint(mx), false, false);
    // in log2 units they are fp16 numbers as they are, but for rows that would leave its normal range: those by a
    // power of two, made good at the scores (of 2^-62 at least: rows smaller than that have no scores to tell apart, and
    // neither factor may become 0 or infinite)
    const float top = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1])) * norm;
    int ex = top > 0x1p-10f && top < 0x1p15f ? 0 : row_exponent(top);
    if (ex < -62) ex = -62;
    qs = ldexpf(1.0f, ex);
    norm = ldexpf(norm, -ex);
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) qf[c][e] = (_Float16)(w[8 * c + kOrder[e]] * norm);
  }
  const bool shifted = !RELATIVE || __builtin_amdgcn_ballot_w64(qs != 1.0f) != 0;

  f32x16 acc[NB];
#pragma unroll
  for (int db = 0; db < NB; ++db)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[db][r] = 0.0f;
  // scores are made relative to m, the running maximum less kLift; with nothing seen yet, to 0
  float m = 0.0f, slack = -__builtin_inff(), l = 0.0f;
  f32x16 minus;
#pragma unroll
  for (int r = 0; r < 16; ++r) minus[r] = 0.0f;

  auto scores = [&](const char* buf, f32x16* s) {
    s[0] = s[1] = minus;
    // the two blocks' sums in turn, so that neither waits for itself
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const half8v a = *reinterpret_cast<const half8v*>(buf + (2 * c + h) * L::KROW + (32 * st + n) * 16);
        s[st] = mma32(a, qf[c], s[st]);
      }
  };
  // Scores of tile t + 1 are made while the softmax works on those of t; keys
  // are a tile ahead of the values, in LDS and on their way.
  f32x16 s[2];
  if (from < to) {
    if (does_k) {
      store_keys<D>(xk0, kbuf, wave & 3, lane);
      store_keys<D>(xk1, kbuf + L::KEYS, wave & 3, lane);
    }
    if (does_v) store_values<D>(xv0, vbuf, wave & 3, lane, from + blk, lo, to);
  }
  __syncthreads();
  if (from < to) scores(kbuf, s);
  __syncthreads();
  int cur = 0;
  for (int t0 = from; t0 < to; t0 += kPromptTokens) {
    const int end = all_hi < to ? all_hi : to;
    if (t0 < all_lo || t0 + kPromptTokens > end) {
      // the row's tokens as bits, one of them spread over a score at a time
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const uint32_t seen = (low_bits(my_end - t0 - 32 * st) & ~low_bits(my_lo - t0 - 32 * st)) >> (4 * h);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const uint32_t k = (uint32_t)__builtin_amdgcn_sbfe(seen, 8 * (r >> 2) + (r & 3), 1);
          s[st][r] = __uint_as_float((__float_as_uint(s[st][r]) & k) | (~k & 0xFF800000u));
        }
      }
    }
    if (shifted) {
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[st][r] = fmaf(s[st][r], qs, -m);
    }
    float mx = s[0][0];
#pragma unroll
    for (int st = 0; st < 2; ++st)
#pragma unroll
      for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[st][r]);
    if (__builtin_amdgcn_ballot_w64(mx > slack)) {
      const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(mx), __float_as_uint(mx), false, false);
      const float up = fmaxf(__uint_as_float(sw[0]), __uint_as_float(sw[1]));
      const bool first = slack < 0.0f, some = up > -__builtin_inff();
      const float by = first ? (some ? up - kLift : 0.0f) : fmaxf(up - kLift, 0.0f);
      const float f = first ? 1.0f : exp2f(-by);
      if (some) slack = kLift + kMaxSlack;
      m += by;
      l *= f;
#pragma unroll
      for (int db = 0; db < NB; ++db) acc[db] *= f;
      s[0] -= by;
      s[1] -= by;
      const float mm = shifted ? 0.0f : -m;
#pragma unroll
      for (int r = 0; r < 16; ++r) minus[r] = mm;
    }
    // what is asked for at the end of this turn; its page id is read early
    const Place pv = ahead;
    ahead = place_of<D>(p.c, table_row, head, t0 + 3 * kPromptTokens + blk, last);

    // the next tile's scores, and this one's probabilities; their sum takes them as rounded, and like the matrix
    // instructions the dot product keeps fp16's subnormals (both checked against exact sums)
    f32x16 sn[2];
    scores(kbuf + (cur ^ 1) * L::KEYS, sn);
    half8v ph[4];
    const half2v one2 = {(_Float16)1, (_Float16)1};
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float e0 = __builtin_amdgcn_exp2f(s[t >> 1][8 * (t & 1) + i]);
        const float e1 = __builtin_amdgcn_exp2f(s[t >> 1][8 * (t & 1) + i + 1]);
        const half2v e = {(_Float16)e0, (_Float16)e1};
        ph[t][i] = e[0];
        ph[t][i + 1] = e[1];
        l = __builtin_amdgcn_fdot2(e, one2, l, false);
      }

    // O^T over four 16-token steps, and the next tiles' codes to LDS
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int db = 0; db < NB; ++db) {
        const half8v a = *reinterpret_cast<const half8v*>(vbuf + cur * L::VALUES + ((2 * t + h) * D + 32 * db + n) * 16);
        acc[db] = mma32(a, ph[t], acc[db]);
      }
    if (does_k) {
      store_keys<D>(xk, kbuf + cur * L::KEYS, wave & 3, lane);
      load_keys<D>(p.c, ahead, lane, xk);
    }
    if (does_v) {
      store_values<D>(xv, vbuf + (cur ^ 1) * L::VALUES, wave & 3, lane, t0 + kPromptTokens + blk, lo, to);
      load_values<D>(p.c, pv, lane, xv);
    }
    s[0] = sn[0];
    s[1] = sn[1];
    cur ^= 1;
    __syncthreads();
  }
  {
    const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
    l = __uint_as_float(sw[0]) + __uint_as_float(sw[1]);
  }
  if (!valid) return;
  // output: lane (h, n) holds dims u NC + c of row n, u = 8 (i / 4) + 4 h + i % 4 (i < 8): turned back as the
  // queries were turned
  float w[D / 2];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int c = 0; c < NC; ++c) w[i * NC + c] = acc[c >> 1][8 * (c & 1) + i];
  const int64_t out_row = (int64_t)(q.s0 + n_mine) * p.q_heads + q_head;
  if (parts > 1 && p.nsplit > 1) {
    const int64_t at = out_row * p.nsplit + part;
#pragma unroll
    for (int i = 0; i < 8; ++i) store_vec<kDtF32, NC>(p.part_o + at * D + (8 * (i >> 2) + 4 * h + (i & 3)) * NC, w + i * NC);
    if (h == 0) p.part_ml[at] = make_float2(slack < 0.0f ? -__builtin_inff() : m, l);
    return;
  }
  float f = l == 0.0f ? 0.0f : 1.0f / l;
  if (p.c.rotate) {
    fwht_halves<D / 2>(w, h);
    f *= kv4_norm<D>();
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int dim = (8 * (i >> 2) + 4 * h + (i & 3)) * NC;
    uint32_t sg[NC];
    if (p.c.rotate) load_signs<NC>(p.c.signs, dim, sg);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      w[i * NC + c] *= f;
      if (p.c.rotate) w[i * NC + c] = flip(w[i * NC + c], sg[c]);
    }
    store_vec<kDtBf16, NC>(reinterpret_cast<uint16_t*>(p.out) + out_row * D + dim, w + i * NC);
  }
}

template <int D, int W>
static void prompt2(const Kv4AttnArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((kv4_prompt_kernel<D, W>), dim3((unsigned)a.groups), dim3(64 * W), 0, s, a);
}

void launch_kv4_prompt(const Kv4AttnArgs& a, hipStream_t s) {
  switch (a.c.dim) {
    case 64: prompt2<64, 4>(a, s); break;
    case 128:
      if (a.rows == 256) prompt2<128, 8>(a, s);
      else prompt2<128, 4>(a, s);
      break;
    default: prompt2<256, 4>(a, s); break;
  }
}

}  // namespace hr
