// Internal declarations shared by the HIP translation units of libhr.so.
// Nothing here is part of the public ABI (include/hr.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hr {

// Inputs at least this large are read with the nontemporal hint.  Streamed
// once from HBM they are faster with it (bf16 65536 x 2048 rotation: 62.9
// against 63.8 us; the rotation-free quantizer 57.4 against 63.8 us); a
// smaller input may still sit in the 256 MB last-level cache from whatever
// wrote it, and the hint then costs (bf16 4096 x 4096 rotation read again
// each call: 14.3 against 12.9 us).  A quarter of that cache, same box.
constexpr int64_t kStreamBytes = int64_t(64) << 20;

// Arguments of one rotate / rotate+quantize call after host validation.
struct RhtArgs {
  const void* x;
  int x_bf16;            // 1: bf16 input, 0: fp32 input
  int64_t rows;
  int n, m, p;           // n = m * p
  const int8_t* signs;   // may be null (all +1)
  const float* block;    // [m][m], null when m == 1
  float* y;              // fp32 output or null
  int group;             // quantization group (when codes != null)
  uint8_t* codes;        // packed int4 (bits 4), int8 (bits 8) or tiled fp6 (bits 6) codes, or null
  int bits;              // 4, 8 or 6 (when codes != null)
  void* scales;          // scale output or null
  int scale_f16;         // 1: fp16 scales, 0: fp32 scales
};

// Arguments of one rotation-free quantize call after host validation.
struct QuantArgs {
  const void* x;
  int x_bf16;            // 1: bf16 input, 0: fp32 input
  int64_t rows;
  int n;                 // a multiple of group
  int group;
  int bits;              // 4 (packed int4 codes) or 8 (int8 codes)
  uint8_t* codes;
  void* scales;
  int scale_f16;
};

struct ButterflyArgs {
  const float* x;
  float* y;
  int64_t rows;
  int n, log2n;
  const float* coeffs;   // [log2 n][n/2][2]
  int precondition;
  const int* perm;
  int inverse;
  int group;
  uint8_t* codes;
  void* scales;
  int scale_f16;
};

struct GemmArgs {
  const uint8_t* a;      // packed int4 [M][K/2], or int8 [M][K] when a_int8
  int a_int8;            // 1: int8 activation codes [M][K] (W4A8, W8A8)
  int w_int8;            // 1: int8 weight codes [N][K] (W8A8)
  const void* sa;
  const uint8_t* w;
  const void* sw;
  int scale_f16;
  int64_t M, N, K;
  int group;
  float* c;
  int32_t* group_acc;
};

// Arguments of the fused decode call (rotation + int4 quantization of M <= 16
// bf16 rows, then the W4A4 GEMM on the codes) after host validation.
struct FusedDecodeArgs {
  const uint16_t* x;     // bf16 [M][K]
  const int8_t* signs;   // [K] or null
  float norm;            // 1 / sqrt(K)
  const uint8_t* w;      // packed int4 [N][K/2]
  const void* sw;        // [N][K/G]
  int scale_f16;
  int64_t M, N, K;
  int group;
  float* c;              // [M][N]
  uint8_t* a_codes;      // optional [M][K/2] copy of the activation codes
  void* a_scales;        // optional [M][K/G] copy of their scales
};

constexpr int kHarpMaxStages = 16;
constexpr int kHarpMaxRadix = 8;

// A mixed-radix schedule with its per-stage offsets (filled on the host).
struct HarpSchedule {
  int nstages;
  int radix[kHarpMaxStages];
  int stride[kHarpMaxStages];               // b_0 ... b_{t-1}
  int64_t block_begin[kHarpMaxStages + 1];  // global index of the first block of each stage
  int64_t theta_off[kHarpMaxStages];        // floats into theta
  int64_t fallback_off[kHarpMaxStages];     // floats into fallbacks (radices not a power of two)
  int64_t blocks_off[kHarpMaxStages];       // floats into the block table
};

struct HarpArgs {
  const float* x;
  float* y;              // fp32 output or null
  int64_t rows;
  int d;
  HarpSchedule sc;
  const float* blocks;
  int inverse;
  int group;
  uint8_t* codes;        // packed int4 output or null
  void* scales;
  int scale_f16;
  int rows_per_group;    // set by the launcher
  int stream;            // set by the launcher: nontemporal row loads
};

// Element types of the key/value cache calls (the values of hr_dtype).
constexpr int kDtF32 = 0, kDtBf16 = 1, kDtF16 = 2;

// Largest cached length: token indices of a sequence stay in 32 bits.
constexpr int kKv4MaxLen = 1 << 30;

// A 4-bit key/value cache after host validation (layout: kv4_device.h).
struct Kv4Cache {
  uint8_t* codes[2];     // keys, values
  _Float16* scales[2];
  const int8_t* signs;   // [dim] or null (all +1; only read with rotate)
  int64_t pages;
  int heads, dim, group;
  int page_log2;
  int rotate;
};

struct Kv4AppendArgs {
  Kv4Cache c;
  const void* x[2];      // keys, values: [tokens] rows of [heads][dim], rows `stride` elements apart
  int64_t stride[2];
  int dtype;
  const int64_t* slots;
  int64_t tokens;
};

struct Kv4ReadArgs {
  Kv4Cache c;
  void* y[2];            // keys, values: [tokens][heads][dim]
  int dtype;
  const int64_t* slots;
  int64_t tokens;
};

struct Kv4AttnArgs {
  Kv4Cache c;
  const void* q;         // [total] rows of [q_heads][dim], rows q_stride elements apart
  int64_t q_stride;
  int dtype;             // of q and out
  int64_t total;
  const int32_t* starts; // [batch + 1] first row of each sequence, or null (max_new rows each)
  const int32_t* table;  // [batch][width] page ids
  int64_t width;
  const int32_t* lens;   // [batch]
  int batch, q_heads, rep;
  int max_new;
  int64_t max_len;
  float scale;
  int causal, window;
  void* out;             // [total][q_heads][dim]
  float* part_o;         // [total * q_heads][nsplit][dim] sums, not yet divided; null when nsplit == 1
  float2* part_ml;       // [total * q_heads][nsplit] (running max in log2 units, sum)
  // by kv4_attention_plan:
  int rows;              // of a row tile: 16, 32, or 128 or 256 (kv4_prompt.hip)
  int waves;             // of a workgroup with 16 rows: 4 or 8
  int tiles;             // row tiles of a (sequence, key/value head)
  int nsplit, chunk;     // most parts of the token axis, tokens of a part
  int64_t groups;        // workgroups
};

hipError_t launch_kv4_append(const Kv4AppendArgs& a, hipStream_t s);
hipError_t launch_kv4_read(const Kv4ReadArgs& a, hipStream_t s);
// Fills its part of the arguments from the sizes and types.
void kv4_attention_plan(Kv4AttnArgs* a);
hipError_t launch_kv4_attention(const Kv4AttnArgs& a, hipStream_t s);
void launch_kv4_prompt(const Kv4AttnArgs& a, hipStream_t s);   // its part when a.rows >= 128

hipError_t launch_harp_blocks(const HarpSchedule& sc, const float* theta, const float* fallbacks,
                              float* blocks, hipStream_t s);
hipError_t launch_harp_apply(HarpArgs a, hipStream_t s);

hipError_t launch_rht(const RhtArgs& a, hipStream_t s);
hipError_t launch_quant(const QuantArgs& a, hipStream_t s);
bool launch_rht2048(const RhtArgs& a, hipStream_t s);  // false: not handled
bool launch_rht2048_mfma(const RhtArgs& a, hipStream_t s);  // false: not handled
bool launch_mixed2048_mfma(const RhtArgs& a, hipStream_t s);  // false: not handled
hipError_t launch_butterfly_coeffs(const float* angles, int n, int log2n, int precondition,
                                   float* coeffs, hipStream_t s);
hipError_t launch_butterfly(const ButterflyArgs& a, hipStream_t s);
bool launch_butterfly4096(const ButterflyArgs& a, hipStream_t s);  // false: not handled
hipError_t launch_dequant(const uint8_t* codes, const void* scales, int scale_f16, int64_t rows,
                          int n, int group, float* out, hipStream_t s);
hipError_t launch_gemm(const GemmArgs& a, hipStream_t s);
// bf16 rows of n = 2048 or 4096, int4 codes in the tiled fp6 format (a.codes)
// and transposed scales (a.scales), G = 128 or 256; false for other cases
bool launch_rotate_quant_fp6(const RhtArgs& a, hipStream_t s);
// scales may be null (then out_scales, scale_f16 and group are unused)
hipError_t launch_int4_to_fp6(const uint8_t* codes, const void* scales, bool scale_f16, int64_t rows, int64_t K,
                              int group, uint8_t* out, void* out_scales, hipStream_t s);
// a.a, a.w: tiled fp6; a.sa, a.sw: transposed scales [K / G][padded rows]
hipError_t launch_gemm_fp6(const GemmArgs& a, hipStream_t s);
hipError_t launch_rotate_quant_gemm_decode(const FusedDecodeArgs& a, hipStream_t s);
bool launch_gemm_mfma(const GemmArgs& a, hipStream_t s);  // false: not handled

}  // namespace hr
