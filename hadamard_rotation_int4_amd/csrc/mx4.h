// What the host side hands to the kernels of the MXFP4 format and of the norms
// between two blocks.
#pragma once

#include "hr_internal.h"

namespace hr {

constexpr int kMxBlock = 32;           // elements of a scale
constexpr int kMxMaxN = 1 << 18;       // longest row that is quantized or read back
constexpr int kNormMaxN = 32768;       // longest row that is normed

// Rows to MXFP4 codes and scales, after host validation.
struct Mx4QuantArgs {
  const void* x;         // [rows] rows of n elements, x_stride apart
  int dtype;             // hr_dtype
  int64_t x_stride;
  int64_t rows;
  int n;
  int order;             // of the Hadamard blocks, 0: no rotation
  const int8_t* signs;   // [n] or null (all +1)
  int ceil;              // scale rule: 1: the largest element never saturates
  uint8_t* codes;        // [rows][n / 2]
  uint8_t* scales;       // [rows][n / 32]
  int stream;            // set by the launcher: nontemporal loads of x
};

struct Mx4DequantArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t rows;
  int n;
  int order;
  const int8_t* signs;
  int dtype;             // of y
  void* y;               // [rows][n]
  int stream;            // set by the launcher: nontemporal stores of y
};

struct Mx4GemmArgs {
  const uint8_t* a;      // [M][K / 2]
  const uint8_t* sa;     // [M][K / 32]
  const uint8_t* w;      // [N][K / 2]
  const uint8_t* sw;     // [N][K / 32]
  int64_t M, N;
  int K;
  int dtype;             // of c
  void* c;               // [M][N]
};

// r = x + scale gate (block or its norm), h = weight r / rms(r), after host
// validation.
struct NormArgs {
  const void* x;         // [rows] of x_dtype, x_stride apart
  const void* block;     // [rows] of dtype, block_stride apart, or null
  const float* post_weight;
  const void* gate;      // [gates] rows of dtype, or null
  const float* weight;
  int64_t x_stride, block_stride, residual_stride;
  int64_t rows, gate_rows;   // gate_rows: rows that share a gate
  int n;
  int x_dtype, dtype;
  int post_norm;
  float scale, eps;
  void* residual;        // of x_dtype, or null
  void* h;               // [rows][n] of dtype, or null
  int order;             // the rest: h as MXFP4 where codes is set
  const int8_t* signs;
  int ceil;
  uint8_t* codes;
  uint8_t* scales;
  float turn;            // set by the launcher: 1 / sqrt(order), 1 without a rotation
};

hipError_t launch_mx4_quant(const Mx4QuantArgs& a, hipStream_t s);
hipError_t launch_mx4_dequant(const Mx4DequantArgs& a, hipStream_t s);
// Their parts where 16-bit rows are rotated.
void launch_mx4_rotate_quant(const Mx4QuantArgs& a, hipStream_t s);
void launch_mx4_rotate_back(const Mx4DequantArgs& a, hipStream_t s);
hipError_t launch_mx4_gemm(const Mx4GemmArgs& a, hipStream_t s);
hipError_t launch_norm(const NormArgs& a, hipStream_t s);
// Its parts by the types of the stream and of the block.
void launch_norm_f16(const NormArgs& a, hipStream_t s);
void launch_norm_f32_bf16(const NormArgs& a, hipStream_t s);
void launch_norm_f32_f16(const NormArgs& a, hipStream_t s);
void launch_norm_f32(const NormArgs& a, hipStream_t s);

}  // namespace hr
