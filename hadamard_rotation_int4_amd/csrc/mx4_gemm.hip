// Product of two MXFP4 operands, C = A W^T, on the matrix cores' scaled fp4
// instructions.
//
// What is computed: C[m][n] = sum over blocks j of 2^(Ea[m][j] + Ew[n][j]) times
// the sum of the 32 products of the block's codes, in fp32, rounded once to
// the output type.
//
// v_mfma_scale_f32_16x16x128_f8f6f4: lane l holds row l % 16 of its operand and
// the 32 codes (16 bytes) of block l / 16 of the step's four, with that block's
// scale byte; the 32x32x64 form likewise with rows l % 32 and two blocks.  The
// weights are the first operand, so that a lane's results are four consecutive
// columns of one row of C at a time.
//
// Rates on random codes: the 32x32x64 instruction alone, nothing loaded, reaches 6.4
// PFLOP/s on the whole card (9.0 on zeros: the clock falls with the power drawn, from
// 2.5 to 1.5 GHz), the 16x16x128 one 5.5.  The 256 x 256 tile reaches 3.9 to 4.1 at 4096 x
// 4096 x 14336 and 3.5 to 3.9 at 8192 x 14336 x 4096 (247 to 272 us by the card), where the
// matrix cores are busy 46% of the clocks, at 1.9 GHz; at 4096^3 (256 tiles, one a compute
// unit) 3.2 to 3.7 PFLOP/s, 38 to 43 us, 7 of them stores at the end and 3 the first loads.
// Of 119 us at 4096 x 4096 x 14336 products alone take 86, the copies into LDS cost 19 (where
// they come from hardly matters: always of one stage, 115) and the reads out of it 14, one
// after another: 192 KB read and 64 written a stage and workgroup are 2048 cycles of LDS, as
// many as its products take, but a stage takes some 4400, for all waves meet at one barrier
// a stage, then read and multiply together.  What was tried on it made no
// difference: other orders of its LDS reads, copies and products, waves' priorities,
// copies spread over the steps, bank conflicts taken out (270 against 272 us), dies starting
// at other stages of K; waves of 64 x 128 instead of 128 x 64 are 1% slower, 4 waves of
// 128 x 128, alone on their SIMDs, 133 against 121 us.
#include "mx4_copy.h"
#include "mx4_device.h"

namespace hr {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kFp4 = 4;      // format code of the instruction's operands

__device__ __forceinline__ v8i fp4_operand(const uint4& x) {
  return (v8i){(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
}

// One element of C, rounded to its type.
__device__ __forceinline__ void store_c(const Mx4GemmArgs& p, int64_t at, float v) {
  if (p.dtype == kDtF32) reinterpret_cast<float*>(p.c)[at] = v;
  else if (p.dtype == kDtBf16) reinterpret_cast<__bf16*>(p.c)[at] = (__bf16)v;
  else reinterpret_cast<_Float16*>(p.c)[at] = (_Float16)v;
}

// 16 bytes of a row of C at any address: four elements in 32 bits, eight in 16; around
// the L2s with NT.
template <bool NT>
__device__ __forceinline__ void store_unit_c(const Mx4GemmArgs& p, int64_t at, const float* v) {
  typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
  u32x4_any x;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (p.dtype == kDtF32) x[e] = __float_as_uint(v[e]);
    else if (p.dtype == kDtBf16) x[e] = __builtin_bit_cast(uint32_t, (bf16x2){(__bf16)v[2 * e], (__bf16)v[2 * e + 1]});
    else x[e] = __builtin_bit_cast(uint32_t, (half2v){(_Float16)v[2 * e], (_Float16)v[2 * e + 1]});
  }
  u32x4_any* q = reinterpret_cast<u32x4_any*>(reinterpret_cast<char*>(p.c) + at * (p.dtype == kDtF32 ? 4 : 2));
  if (NT) __builtin_nontemporal_store(x, q);
  else *q = x;
}

// 16 columns and 16 MT rows of C a workgroup.  K goes in runs of 512 codes (four
// steps of 128: 256 bytes of a row and 16 of its scales), which the waves take in
// turn straight from memory into registers, all loads of a run before its products;
// their sums are joined in LDS, in the waves' order.
template <int MT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void mx4_gemm_rows_kernel(Mx4GemmArgs p) {
  struct __attribute__((packed, aligned(1))) Scales { uint32_t v[4]; };
  __shared__ v4f part[WAVES][MT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, kb = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * (16 * MT);
  const int blocks = p.K / kMxBlock, runs = blocks / 16;
  // rows past the end: the last again, stored nowhere
  const int64_t wrow = n0 + r < p.N ? n0 + r : p.N - 1;
  const uint8_t* const w = p.w + wrow * (p.K / 2) + 16 * kb;
  const uint8_t* const sw = p.sw + wrow * blocks;
  const uint8_t* a[MT];
  const uint8_t* sa[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int64_t row = m0 + 16 * t + r < p.M ? m0 + 16 * t + r : p.M - 1;
    a[t] = p.a + row * (p.K / 2) + 16 * kb;
    sa[t] = p.sa + row * blocks;
  }
  v4f acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
  struct Run {
    uint4 wc[4], ac[MT][4];
    Scales ws, as[MT];
  };
  auto load = [&](int q, Run& x) {
#pragma unroll
    for (int s = 0; s < 4; ++s) x.wc[s] = *reinterpret_cast<const uint4*>(w + 256 * q + 64 * s);
    x.ws = *reinterpret_cast<const Scales*>(sw + 16 * q);
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
      for (int s = 0; s < 4; ++s) x.ac[t][s] = *reinterpret_cast<const uint4*>(a[t] + 256 * q + 64 * s);
      x.as[t] = *reinterpret_cast<const Scales*>(sa[t] + 16 * q);
    }
  };
  auto multiply = [&](const Run& x) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int t = 0; t < MT; ++t)
        acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(x.wc[s]), fp4_operand(x.ac[t][s]), acc[t], kFp4,
                                                                  kFp4, 0, (int)(x.ws.v[s] >> (8 * kb)), 0,
                                                                  (int)(x.as[t].v[s] >> (8 * kb)));
  };
  if (MT == 1) {
    // the next three runs are under way while one is multiplied (16 x 4096 x 14336, 3.5 runs
    // a wave: 11.0 us, with one 11.9, two 11.1, four 10.9)
    constexpr int AHEAD = 3;
    Run x[AHEAD + 1];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (wave + i * WAVES < runs) load(wave + i * WAVES, x[i]);
    for (int q = wave; q < runs; q += (AHEAD + 1) * WAVES) {
#pragma unroll
      for (int i = 0; i <= AHEAD; ++i) {
        const int at = q + i * WAVES;
        if (at >= runs) break;
        if (at + AHEAD * WAVES < runs) load(at + AHEAD * WAVES, x[(i + AHEAD) % (AHEAD + 1)]);
        __builtin_amdgcn_sched_barrier(0);
        multiply(x[i]);
      }
    }
  } else {
    for (int q = wave; q < runs; q += WAVES) {
      Run x;
      load(q, x);
      multiply(x);
    }
  }
  // what is left of K: fewer than four steps, past its end zero codes and scales
  if (wave == runs % WAVES) {
    for (int j = 16 * runs + kb; j < blocks + kb; j += 4) {
      const bool live = j < blocks;
      const uint4 z = make_uint4(0u, 0u, 0u, 0u);
      const uint4 wc = live ? *reinterpret_cast<const uint4*>(w + 16 * (j - kb)) : z;
      const int ws = live ? sw[j] : 0;
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const uint4 ac = live ? *reinterpret_cast<const uint4*>(a[t] + 16 * (j - kb)) : z;
        const int as = live ? sa[t][j] : 0;
        acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(wc), fp4_operand(ac), acc[t], kFp4, kFp4, 0, ws,
                                                                  0, as);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) part[wave][t][lane] = acc[t];
  __syncthreads();
  const bool quads = p.N % 4 == 0;
  for (int i = threadIdx.x; i < MT * 64; i += 64 * WAVES) {
    const int t = i >> 6, l = i & 63;
    v4f c = part[0][t][l];
#pragma unroll
    for (int v = 1; v < WAVES; ++v) c += part[v][t][l];
    const int64_t m = m0 + 16 * t + (l & 15), n = n0 + 4 * (l >> 4);
    if (m >= p.M) continue;
    const float x[4] = {c[0], c[1], c[2], c[3]};
    if (quads) {
      if (n < p.N) store_vec_any<4>(p.dtype, p.c, m * p.N + n, x);
    } else {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (n + v < p.N) store_c(p, m * p.N + n + v, x[v]);
    }
  }
}

// ---------------------------------------------------------------- tiles

template <int V>
struct MxC { static constexpr int value = V; };

constexpr int kSchedMfma = 0x8, kSchedDsRead = 0x100;

// (32 WM TM) x (32 WN TN) outputs a workgroup of WM WN waves, TM x TN tiles of
// v_mfma_scale_f32_32x32x64_f8f6f4 a wave.
//
// A stage is 256 codes of K: 128 bytes of each row, copied from memory into LDS
// (8 rows an instruction), D stages in LDS: a stage of a small tile takes less time than
// its copies are under way, so that D - 1 of them are at a time.  A lane of the instruction holds
// row l % 32 of its operand and 32 codes; half h = l / 32 takes blocks 4 h + s at
// step s < 4 of a stage, so that one 4-byte word holds a lane's scales of the
// stage and the step picks its byte.  In LDS the 16-byte chunk c of row r sits
// at chunk c ^ (r / 2 % 8): 16 consecutive rows of one chunk, which a read serves at
// once, lie in the 16 places of 256 bytes (with r % 8 two and two met, 4 cycles a
// read).  The copy writes LDS in lane order, so it is the source chunk of a lane that
// is permuted, within the row's 128 bytes.
//
// SM, how a lane gets its scales.  kCopied: copied into LDS, 16 bytes of each row
// every second stage, where each row's are whole runs of 16.  kBrought: the same
// through registers, at any alignment, for K of at least 512.  kOwn: each lane loads
// its own words, for K of at least 128.  kFew: its own bytes, for fewer than four blocks.
//
// KG: teams of WM WN waves that take pairs of stages in turn, each with buffers of
// its own; their sums are joined in LDS, in the teams' order.  For the smallest tiles,
// of which a workgroup would else be one or two waves.
enum { kOwn, kCopied, kBrought, kFew };

template <int WM, int WN, int TM, int TN, int KG, int D, int SM, int OCC, bool NT>
__global__ __launch_bounds__(64 * WM * WN * KG, OCC) void mx4_gemm_tile_kernel(Mx4GemmArgs p, int tiles_m, int tiles_n) {
  constexpr int WAVES = WM * WN, BM = 32 * WM * TM, BN = 32 * WN * TN, T = TM + TN;
  constexpr int ROWB = kMxStageBytes;              // bytes of a row and stage
  constexpr int QA = BM / 8, QW = BN / 8;          // copies of 1 KB of a stage
  constexpr int DPW = (QA + QW) / WAVES;
  constexpr bool SL = SM == kCopied || SM == kBrought;             // through LDS
  constexpr int SA = (BM + 63) / 64, QS = SA + (BN + 63) / 64;     // copies of 64 rows' scales of two stages
  constexpr int SCB = SM == kCopied ? QS * 1024 : SL ? (BM + BN) * 16 : 16;      // bytes of them
  constexpr int SPW = (QS + WAVES - 1) / WAVES;    // copies of a wave
  constexpr int SPT = (BM + BN + 64 * WAVES - 1) / (64 * WAVES);   // rows of scales of a thread
  constexpr int BUF = (BM + BN) * ROWB;
  static_assert((QA + QW) % WAVES == 0 && DPW % 2 == 0 && QA % 2 == 0, "equal copies a wave, even and odd ones known");
  // arrays of their own, so that a read is known not to wait for copies into others
  __shared__ __attribute__((aligned(16))) char sbuf0[KG * BUF];
  __shared__ __attribute__((aligned(16))) char sbuf1[KG * BUF];
  __shared__ __attribute__((aligned(16))) char sbuf2[D > 2 ? KG * BUF : 16];
  __shared__ __attribute__((aligned(16))) char sbuf3[D > 2 ? KG * BUF : 16];
  __shared__ __attribute__((aligned(16))) char sscale0[(D > 2 ? 1 : 2) * KG * SCB];
  __shared__ __attribute__((aligned(16))) char sscale1[D > 2 ? KG * SCB : 16];
  const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
  const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int team = KG == 1 ? 0 : wave_all / WAVES, wave = wave_all - team * WAVES;
  const int wm = wave / WN * (32 * TM), wn = wave % WN * (32 * TN);

  // Workgroups go round the 8 dies in turn: each die takes a run of consecutive
  // tiles, which go down 8 rows of tiles before the next column, so that the
  // dies' L2s share panels of both operands.
  const int total = tiles_m * tiles_n, die = blockIdx.x & 7;
  const int tile = die * (total >> 3) + min(die, total & 7) + (int)(blockIdx.x >> 3);
  const int width = 8 * tiles_n, group = tile / width, in = tile - group * width;
  const int high = min(8, tiles_m - 8 * group);
  const int64_t m0 = (int64_t)(8 * group + in % high) * BM, n0 = (int64_t)(in / high) * BN;

  const int blocks = p.K / kMxBlock, stages = mx4_stages(blocks), stride = p.K / 2;
  const int rows_a = (int)(p.M - m0 < BM ? p.M - m0 : BM), rows_w = (int)(p.N - n0 < BN ? p.N - n0 : BN);
  // rows past the end lie past the buffer's end (mx4_copy.h): nothing is read there, and
  // what LDS holds for them (codes are finite whatever they are) goes into outputs
  // that are not stored
  const __amdgpu_buffer_rsrc_t ra =
      __builtin_amdgcn_make_buffer_rsrc((void*)(p.a + m0 * stride), 0, rows_a * stride, 0x00020000);
  const __amdgpu_buffer_rsrc_t rw =
      __builtin_amdgcn_make_buffer_rsrc((void*)(p.w + n0 * stride), 0, rows_w * stride, 0x00020000);
  // of even and odd copies; in the last stage chunks past the end take the row's last
  // one (under zero scales)
  int src[2], src_last[2];
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    src[o] = mx4_lane_offset(lane, o, blocks);
    src_last[o] = mx4_lane_offset_last(lane, o, blocks);
  }
  auto buf = [&](auto b) -> char* {
    constexpr int B = decltype(b)::value;
    if constexpr (B == 0) return sbuf0 + team * BUF;
    else if constexpr (B == 1) return sbuf1 + team * BUF;
    else if constexpr (B == 2) return sbuf2 + team * BUF;
    else return sbuf3 + team * BUF;
  };
  // the scales of the team's stages 2 i and 2 i + 1 (i odd or even known where D > 2)
  auto slot = [&](int i, auto odd) -> char* {
    if constexpr (D == 2) return sscale0 + (i & 1) * (KG * SCB) + team * SCB;
    else if constexpr (decltype(odd)::value == 0) return sscale0 + team * SCB;
    else return sscale1 + team * SCB;
  };
  // the team's stage i as a stage of K
  auto place = [&](int i) { return KG == 1 ? i : 2 * (KG * (i >> 1) + team) + (i & 1); };
  // stage s into buffer b; behind the last stage nothing is read (the loop has no
  // branch: the compiler would move products over it)
  auto copy = [&](int s, auto b) {
    char* dst = buf(b);
    int v[2];
#pragma unroll
    for (int o = 0; o < 2; ++o) v[o] = mx4_stage_offset(s, stages, src[o], src_last[o]);
#pragma unroll
    for (int j = 0; j < DPW; ++j) {
      const int q = wave * DPW + j;
      const bool a = q < QA;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(a ? ra : rw,
                                               (__attribute__((address_space(3))) void*)(dst + 1024 * q), 16,
                                               mx4_copy_offset(v[j & 1], 8 * (a ? q : q - QA), blocks), s * ROWB, 0, 0);
    }
  };

  // Scales: the 4-byte word of blocks 8 s + 4 h .. + 3 of each of this lane's rows.
  // Past the end of a row words are zero.  A zero byte is 2^-127, and in both
  // operands its products are below 2^-240 and count as 0 whatever the codes are.
  struct __attribute__((packed, aligned(1))) Word { uint32_t v; };
  struct __attribute__((packed, aligned(1))) Run { uint32_t v[4]; };
  const uint8_t* const sa = p.sa + m0 * blocks;
  const uint8_t* const sw = p.sw + n0 * blocks;
  // of this stage; of the next (SL: of two; kOwn: of the stages under way)
  uint32_t sc[T], sn[SL ? 1 : D][SL ? 2 * T : T], srow[T];
#pragma unroll
  for (int i = 0; i < T; ++i) {
    const int r = i < TM ? wm + 32 * i + l32 : wn + 32 * (i - TM) + l32;
    if (SL) srow[i] = (uint32_t)(i < TM ? r : (SM == kCopied ? 64 * SA : BM) + r) * 16;
    else srow[i] = (uint32_t)min(r, (i < TM ? rows_a : rows_w) - 1) * blocks;
  }
  // kCopied: of the team's stages 2 i and 2 i + 1; nothing is read behind the end of the
  // operand or of K
  auto copy_scales = [&](int i, auto odd) {
    const int q = KG * i + team;
#pragma unroll
    for (int j = 0; j < SPW; ++j) {
      // where waves are more than copies some make the same one
      const int c = (wave * SPW + j) % QS;
      const bool a = c < SA;
      const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(a ? sa : sw), 0, (a ? rows_a : rows_w) * blocks, 0x00020000);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)(slot(i, odd) + 1024 * c), 16,
                                               mx4_scale_offset(lane, 64 * (a ? c : c - SA), q, blocks), 16 * q, 0, 0);
    }
  };
  // kBrought: a thread brings 16 bytes of its rows, of the team's stages 2 i and 2 i +
  // 1; the last ones, which may be fewer, are made once.
  const uint8_t* run_row[SPT];
  uint32_t run_at[SPT];
  v4u run[SPT], run_last[SPT];
  const int runs = (blocks + 15) / 16;
  if constexpr (SM == kBrought) {
#pragma unroll
    for (int t = 0; t < SPT; ++t) {
      const int r = min((int)threadIdx.x - team * 64 * WAVES + t * 64 * WAVES, BM + BN - 1);     // the last again
      run_row[t] = r < BM ? sa + (int64_t)min(r, rows_a - 1) * blocks : sw + (int64_t)min(r - BM, rows_w - 1) * blocks;
      run_at[t] = (uint32_t)r * 16;
      // the last 16 of the row, shifted down to where the last run begins
      const int down = 16 * runs - blocks;
      const Run x = *reinterpret_cast<const Run*>(run_row[t] + blocks - 16);
      const uint64_t lo = x.v[0] | (uint64_t)x.v[1] << 32, hi = x.v[2] | (uint64_t)x.v[3] << 32;
      const int b = 8 * (down & 7);
      const uint64_t s0 = b ? lo >> b | hi << (64 - b) : lo, s1 = hi >> b;
      const uint64_t y0 = down >= 8 ? s1 : s0, y1 = down >= 8 ? 0 : s1;
      run_last[t] = (v4u){(uint32_t)y0, (uint32_t)(y0 >> 32), (uint32_t)y1, (uint32_t)(y1 >> 32)};
    }
  }
  auto bring_scales = [&](int i) {
    const int q = KG * i + team;
#pragma unroll
    for (int t = 0; t < SPT; ++t) {
      const Run x = *reinterpret_cast<const Run*>(run_row[t] + 16 * min(q, blocks / 16 - 1));
      run[t] = (v4u){x.v[0], x.v[1], x.v[2], x.v[3]};
    }
  };
  auto put_scales = [&](int i, auto odd) {
    const int q = KG * i + team;
#pragma unroll
    for (int t = 0; t < SPT; ++t) {
      v4u x;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = q < runs - 1 ? run[t][e] : q < runs ? run_last[t][e] : 0u;
      *reinterpret_cast<v4u*>(slot(i, odd) + run_at[t]) = x;
    }
  };
  // of the team's stage k; SL: of k, which is even, and k + 1, 16 bytes of a row at once
  auto load_scales = [&](int k, auto odd, uint32_t* v) {
    if constexpr (SL) {
#pragma unroll
      for (int i = 0; i < T; ++i) {
        const v4u x = *reinterpret_cast<const v4u*>(slot(k >> 1, odd) + srow[i]);
        const uint32_t x0 = h ? x[1] : x[0], x1 = h ? x[3] : x[2];
        v[2 * i] = SM == kCopied && 8 * place(k) + 4 * h >= blocks ? 0u : x0;
        v[2 * i + 1] = SM == kCopied && 8 * place(k + 1) + 4 * h >= blocks ? 0u : x1;
      }
    } else if constexpr (SM == kFew) {
#pragma unroll
      for (int i = 0; i < T; ++i) {
        const uint8_t* s = (i < TM ? sa : sw) + srow[i];
        const uint32_t b0 = s[0], b1 = s[min(1, blocks - 1)], b2 = s[blocks - 1];
        v[i] = place(k) > 0 || h ? 0u : b0 | (blocks > 1 ? b1 << 8 : 0u) | (blocks > 2 ? b2 << 16 : 0u);
      }
    } else {
      // past the end of a row its last word, shifted by use_scales
      const uint32_t from = min(8 * place(k) + 4 * h, blocks - 4);
#pragma unroll
      for (int i = 0; i < T; ++i) v[i] = reinterpret_cast<const Word*>((i < TM ? sa : sw) + (srow[i] + from))->v;
    }
  };
  auto use_scales = [&](int k, auto odd, const uint32_t* v) {
    if constexpr (SL) {
#pragma unroll
      for (int i = 0; i < T; ++i) sc[i] = v[2 * i + decltype(odd)::value];
    } else if constexpr (SM == kFew) {
#pragma unroll
      for (int i = 0; i < T; ++i) sc[i] = v[i];
    } else {
      const int half = 4 * min(max(8 * place(k) + 4 * h - (blocks - 4), 0), 4);      // in two shifts: they may be 32 together
#pragma unroll
      for (int i = 0; i < T; ++i) sc[i] = v[i] >> half >> half;
    }
  };

  typedef float v16f __attribute__((ext_vector_type(16)));
  v16f acc[TN][TM];
#pragma unroll
  for (int j = 0; j < TN; ++j)
#pragma unroll
    for (int i = 0; i < TM; ++i) acc[j][i] = (v16f){};

  int at[4];                       // of chunk 4 h + s of this lane's row in a tile
#pragma unroll
  for (int s = 0; s < 4; ++s) at[s] = l32 * ROWB + 16 * ((4 * h + s) ^ ((l32 >> 1) & 7));
  auto read = [&](auto b, int s, uint4 (&f)[T]) {
    const char* base = buf(b);
#pragma unroll
    for (int i = 0; i < TM; ++i) f[i] = *reinterpret_cast<const uint4*>(base + at[s] + (wm + 32 * i) * ROWB);
#pragma unroll
    for (int j = 0; j < TN; ++j) f[TM + j] = *reinterpret_cast<const uint4*>(base + at[s] + (BM + wn + 32 * j) * ROWB);
  };
  auto multiply = [&](auto sc_, const uint4 (&f)[T]) {
    constexpr int S = decltype(sc_)::value;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j)
        acc[j][i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(f[TM + j]), fp4_operand(f[i]), acc[j][i],
                                                                    kFp4, kFp4, S, (int)sc[TM + j], S, (int)sc[i]);
  };
  auto interleave = [&]() {
#pragma unroll
    for (int i = 0; i < T; ++i) {
      __builtin_amdgcn_sched_group_barrier(kSchedDsRead, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kSchedMfma, TM * TN / T > 0 ? TM * TN / T : 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  uint4 f0[T], f1[T];
  // Copies of this wave that may be under way when the next stage has landed.
  constexpr int AWAY = mx4_away(D, DPW, SM == kCopied ? SPW : 0), AWAY0 = mx4_away_first(D, DPW, SM == kCopied ? SPW : 0);
  static_assert(AWAY0 < 64, "vmcnt's six bits");
  constexpr int WAIT = 0x0070 | (AWAY & 15) | (AWAY >> 4) << 14;      // vmcnt(AWAY) lgkmcnt(0)
  // the team's stage k from buffer B: the fragments of its first step are in f0
  auto stage = [&](int k, auto b) {
    constexpr int B = decltype(b)::value, NEXT = (B + 1) % D;
    if (!SL) load_scales(k + D - 1, MxC<0>{}, sn[SL ? 0 : (B + D - 1) % D]);
    read(b, 1, f1);
    multiply(MxC<0>{}, f0);
    interleave();
    read(b, 2, f0);
    multiply(MxC<1>{}, f1);
    interleave();
    read(b, 3, f1);
    multiply(MxC<2>{}, f0);
    interleave();
    // every read of this buffer is done and the next stage has landed, in every wave
    __builtin_amdgcn_s_waitcnt(WAIT);
    mx_barrier();
    if (SL && B % 2 == 1) load_scales(k + 1, MxC<NEXT / 2 % 2>{}, sn[0]);
    read(MxC<NEXT>{}, 0, f0);                      // behind the last stage: nothing uses it
    if (SM == kBrought && B % 2 == 0) {
      // where the scales lay that were read behind the barrier of stage k - 3
      put_scales((k >> 1) + 1, MxC<(B / 2 + 1) % 2>{});
      bring_scales((k >> 1) + 2);
    }
    copy(place(k + D), b);
    // where the scales lay that were read behind the barrier of stage k - 1 (D = 2: k - 3)
    if (SM == kCopied && B % 2 == 0) copy_scales((k >> 1) + D / 2, MxC<(B + D) / 2 % 2>{});
    multiply(MxC<3>{}, f1);
    interleave();
    use_scales(k + 1, MxC<NEXT % 2>{}, sn[SL ? 0 : NEXT]);
  };

  // Copies go out in the order in which stages take them: the waits count on it, and nothing
  // else would keep the compiler to it, as they write arrays of their own.
  auto fence = [&]() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  if constexpr (!SL) load_scales(0, MxC<0>{}, sn[0]);
  copy(place(0), MxC<0>{});
  if constexpr (SM == kCopied) {
    copy_scales(0, MxC<0>{});
  } else if constexpr (SM == kBrought) {
    bring_scales(0);
    put_scales(0, MxC<0>{});
  }
  fence();
  copy(place(1), MxC<1>{});
  fence();
  if constexpr (SM == kBrought) bring_scales(1);
  if constexpr (D > 2) {
    if constexpr (SM == kOwn) load_scales(1, MxC<0>{}, sn[1]);
    fence();
    copy(place(2), MxC<2>{});
    if constexpr (SM == kCopied) copy_scales(1, MxC<1>{});
    if constexpr (SM == kOwn) load_scales(2, MxC<0>{}, sn[2]);
    fence();
    copy(place(3), MxC<3>{});
    fence();
  }
  __builtin_amdgcn_s_waitcnt(0x0070 | (AWAY0 & 15) | (AWAY0 >> 4) << 14);
  mx_barrier();
  if (SL) load_scales(0, MxC<0>{}, sn[0]);
  use_scales(0, MxC<0>{}, sn[0]);
  read(MxC<0>{}, 0, f0);
  // every team runs the same number: behind the end of K under zero scales
  const int turns = KG == 1 ? stages : (stages + 2 * KG - 1) / (2 * KG) * 2;
  int k = 0;
  for (; k + D <= turns; k += D) {
    stage(k, MxC<0>{});
    stage(k + 1, MxC<1>{});
    if constexpr (D > 2) {
      stage(k + 2, MxC<2>{});
      stage(k + 3, MxC<3>{});
    }
  }
  if (k < turns) {
    stage(k, MxC<0>{});
    if constexpr (D > 2) {
      if (k + 1 < turns) stage(k + 1, MxC<1>{});
      if (k + 2 < turns) stage(k + 2, MxC<2>{});
    }
  }
  // no copy is left when LDS is written again or goes to another workgroup
  __builtin_amdgcn_s_waitcnt(0x0070);
  mx_barrier();

  constexpr int PER = WAVES * TM * TN * 4096, FIT = KG * BUF / PER;      // bytes of a team's sums; teams in a buffer
  if constexpr (KG > 1) {
    // the sums of the teams but the first, [wave][tile][quad][lane]
    static_assert(KG - 1 <= 2 * FIT, "fits where the stages were");
    auto part = [&](int g, int i, int j, int q) {
      char* base = g <= FIT ? sbuf0 + (g - 1) * PER : sbuf1 + (g - 1 - FIT) * PER;
      return reinterpret_cast<v4f*>(base + ((((wave * TM + i) * TN + j) * 4 + q) * 64 + lane) * 16);
    };
    if (team > 0) {
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *part(team, i, j, q) =
                (v4f){acc[j][i][4 * q], acc[j][i][4 * q + 1], acc[j][i][4 * q + 2], acc[j][i][4 * q + 3]};
    }
    __syncthreads();
    if (team > 0) return;
#pragma unroll
    for (int g = 1; g < KG; ++g)
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const v4f x = *part(g, i, j, q);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[j][i][4 * q + e] += x[e];
          }
  }

  // A lane holds row l32 of a tile and columns 8 (v / 4) + 4 h + v % 4.  A wave turns
  // 32 rows of its columns at a time in its own part of LDS, so that rows are stored
  // whole; 16-byte unit u of row r at u ^ (r % 8).
  constexpr int CW = 32 * TN, PITCH = CW * 4;
  // with teams behind what they left, which other waves may still be reading
  constexpr int LEFT0 = (KG - 1 < FIT ? KG - 1 : FIT) * PER, SKIP1 = KG - 1 > FIT ? (KG - 1 - FIT) * PER : 0;
  constexpr int HALF = SKIP1 ? 0 : (KG * BUF - LEFT0) / (32 * PITCH);      // waves whose part fits in the first buffer
  static_assert(HALF >= WAVES || SKIP1 + (WAVES - HALF) * 32 * PITCH <= KG * BUF, "fits where the stages were");
  char* const part = wave < HALF ? sbuf0 + LEFT0 + wave * (32 * PITCH) : sbuf1 + SKIP1 + (wave - HALF) * (32 * PITCH);
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<v4f*>(part + l32 * PITCH + 16 * ((8 * j + 2 * q + h) ^ (l32 & 7))) =
            (v4f){acc[j][i][4 * q], acc[j][i][4 * q + 1], acc[j][i][4 * q + 2], acc[j][i][4 * q + 3]};
    __builtin_amdgcn_wave_barrier();
    auto store_rows = [&](auto unit) {
      constexpr int U = decltype(unit)::value, LPR = CW / U;       // elements of a lane, lanes of a row
#pragma unroll
      for (int r = 0; r < 32; r += 64 / LPR) {
        const int rr = r + lane / LPR, n = U * (lane % LPR), m = wm + 32 * i + rr;
        float v[8];
#pragma unroll
        for (int q = 0; q < U / 4; ++q) {
          const v4f x = *reinterpret_cast<const v4f*>(part + rr * PITCH + 16 * ((n / 4 + q) ^ (rr & 7)));
#pragma unroll
          for (int e = 0; e < 4; ++e) v[4 * q + e] = x[e];
        }
        const int64_t to = (m0 + m) * p.N + n0 + wn + n;
        const int left = m < rows_a ? rows_w - wn - n : 0;
        if (left >= U) {
          store_unit_c<NT>(p, to, v);
        } else {
#pragma unroll 1
          for (int e = 0; e < left; ++e)
            store_c(p, to + e, *reinterpret_cast<const float*>(part + rr * PITCH + 16 * (((n + e) / 4) ^ (rr & 7)) + 4 * (e % 4)));
        }
      }
    };
    if (p.dtype == kDtF32) store_rows(MxC<4>{});
    else store_rows(MxC<8>{});
    __builtin_amdgcn_wave_barrier();
  }
}

template <int WM, int WN, int TM, int TN, int KG, int D, int SM, int OCC, bool NT = false>
static void launch_tile(const Mx4GemmArgs& a, hipStream_t s) {
  constexpr int BM = 32 * WM * TM, BN = 32 * WN * TN;
  const int tm = (int)((a.M + BM - 1) / BM), tn = (int)((a.N + BN - 1) / BN);
  hipLaunchKernelGGL((mx4_gemm_tile_kernel<WM, WN, TM, TN, KG, D, SM, OCC, NT>), dim3((unsigned)(tm * tn)),
                     dim3(64 * WM * WN * KG), 0, s, a, tm, tn);
}

template <int MT, int WAVES>
static void launch_rows(const Mx4GemmArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((mx4_gemm_rows_kernel<MT, WAVES>), dim3((unsigned)((a.N + 15) / 16), (unsigned)((a.M + 16 * MT - 1) / (16 * MT))),
                     dim3(64 * WAVES), 0, s, a);
}

// Which tile, by how many of them there are for the 256 compute units: the largest of
// which there is about one for each (kEnough), a few idle units costing less than
// smaller tiles' traffic.  Up to one for each keeps four stages in LDS; more of the larger
// tiles share the units, two and more at a time, and keep two.  64 x 64 and 32 x 64 keep
// four however many they are: two of them share a unit all the same, and long rows gain
// what short ones lose (64 x 64, 1100 x 1111 (324) x 4096 12.6 against 13.1 with two, x
// 1024 7.2 against 6.9; 32 x 64, 30 x 20000 (313) x 4096 15.6 against 17.1, x 1024 6.2 against
// 6.0).  Past one for each 32 x 64 has one team, whose waves alone are enough (two teams
// 17.4, x 1024 8.5).  bf16, us, chosen | next smaller | next larger:
//   256 x 256  1024 x 14336 x 4096 (224) 34 | 42 | -;         3000 x 5120 x 5120 (240) 43 | 52 | -
//   128 x 128  512 x 8192 x 8192 (256) 31 | 44 | 64;          512 x 14336 x 4096 (448) 30 | 43 | 37
//   128 x 64   512 x 4096 x 4096 (256) 11.7 | 13.1 | 14.5;    600 x 4096 x 4096 (320) 14.4 | 17.1 | 15.9
//   64 x 64    256 x 4096 x 4096 (256) 7.9 | 9.6 | 10.7;      40 x 10000 x 4096 (157) 10.4 | 12.3 | 11.2
//   32 x 64    128 x 4096 x 4096 (256) 6.9 | 7.1 | 7.7
//   32 x 32    64 x 4096 x 4096 (256) 5.5 | - | 6.7
// Four stages in LDS against two: 512 x 8192 x 8192 31 against 38, 256 x 4096 x 4096 7.9
// against 11.4; two with more than one tile a unit: 512 x 14336 x 4096 30 against 35.
constexpr int kCus = 256;
constexpr int kEnough = 180, kEnough64 = 140;

// Scales of rows that are not whole runs of 16: through registers into LDS where stages
// are many and waves share them (4096 x 4096 x 4128 54 us against 65, 850 x 900 x 4128
// 10.9 against 11.5), each lane its own where not (850 x 900 x 544 5.0 against 5.3, 64 x
// 4096 x 4128 in teams 7.0 against 7.6).  Whole words could be copied as well, but the
// last 16 bytes would pass the operand's end (4096 x 4096 x 4224 48.9 us instead of 51.0,
// 512 x 4096 x 1152 7.2 instead of 7.6, 512 x 4096 x 640 the same 6.2).
template <int WM, int WN, int TM, int TN, int KG, int D, int OCC, bool NT = false>
static void launch_scales(const Mx4GemmArgs& a, hipStream_t s) {
  // (copies of 16 bytes begin at whole words)
  const bool whole = a.K % 512 == 0 && ((reinterpret_cast<uintptr_t>(a.sa) | reinterpret_cast<uintptr_t>(a.sw)) & 3u) == 0;
  if (whole) launch_tile<WM, WN, TM, TN, KG, D, kCopied, OCC, NT>(a, s);
  else if (KG == 1 && a.K >= 1024) launch_tile<WM, WN, TM, TN, KG, D, KG == 1 ? kBrought : kOwn, OCC, NT>(a, s);
  else launch_tile<WM, WN, TM, TN, KG, D, kOwn, OCC, NT>(a, s);
}

static void launch_tiles(const Mx4GemmArgs& a, hipStream_t s) {
  auto count = [&](int bm, int bn) { return ((a.M + bm - 1) / bm) * ((a.N + bn - 1) / bn); };
  // enough of them, and more than half of one filled either way
  auto fit = [&](int bm, int bn, int enough) { return count(bm, bn) >= enough && 2 * a.M > bm && 2 * a.N > bn; };
  if (a.K < 128) {
    if (fit(128, 128, kEnough)) launch_tile<2, 2, 2, 2, 1, 2, kFew, 2>(a, s);
    else if (fit(64, 64, kEnough64)) launch_tile<2, 2, 1, 1, 1, 2, kFew, 4>(a, s);
    else launch_rows<4, 8>(a, s);
    return;
  }
  // also where 128 x 128 tiles would begin a third round (two a unit): 1400 x 7000 x 4096 (168)
  // 37 us against 45, 1100 x 7680 x 4096 (150) 36 against 39
  if (fit(256, 256, kEnough) || (count(128, 128) > 2 * kCus && fit(256, 256, kCus / 2))) {
    // a large C in 16 bits around the L2s, where the operands are read for long and rows
    // are whole lines: 8192 x 14336 x 4096 265 us against 271 (x 128 69 against 61; in 32 bits
    // 4096 x 8192 x 4096 95 against 87; rows of 14335 x 256 109 against 77)
    if (a.dtype != kDtF32 && a.M * a.N * 2 >= kStreamBytes && a.K >= 2048 && a.N % 64 == 0)
      launch_scales<2, 4, 4, 2, 1, 2, 1, true>(a, s);
    else
      launch_scales<2, 4, 4, 2, 1, 2, 1>(a, s);
  } else if (fit(128, 128, kEnough)) {
    if (count(128, 128) <= kCus) launch_scales<2, 2, 2, 2, 1, 4, 1>(a, s);
    else launch_scales<2, 2, 2, 2, 1, 2, 2>(a, s);
  } else if (fit(128, 64, kEnough)) {
    if (count(128, 64) <= kCus) launch_scales<2, 2, 2, 1, 1, 4, 1>(a, s);
    else launch_scales<2, 2, 2, 1, 1, 2, 2>(a, s);
  } else if (fit(64, 64, kEnough64)) {
    launch_scales<2, 2, 1, 1, 1, 4, 2>(a, s);
  } else if (count(32, 64) >= kEnough && 2 * a.N > 64) {
    if (count(32, 64) <= kCus) launch_scales<1, 2, 1, 1, 2, 4, 1>(a, s);
    else launch_scales<1, 2, 1, 1, 1, 4, 1>(a, s);
  } else {
    launch_scales<1, 1, 1, 1, 2, 4, 1>(a, s);
  }
}

hipError_t launch_mx4_gemm(const Mx4GemmArgs& a, hipStream_t s) {
  // A few rows are bound by the weights' bytes, which go straight to registers while
  // there is a workgroup for each compute unit: 16 x 4096 x 14336 11.0 us (32 x 32 tiles
  // 12.8), one row 8.9, operands past the caches.  With more columns tiles read the rows of
  // A less often: 16 x 8192 x 8192 10.2 us in 32 x 32 tiles, 14.4 in rows (one row of more
  // columns was not measured both ways: 1 x 14336 x 4096 9.9 us in tiles).
  if (a.M <= 16 && a.N <= 4096) launch_rows<1, 8>(a, s);
  else launch_tiles(a, s);
  return hipGetLastError();
}

}  // namespace hr
